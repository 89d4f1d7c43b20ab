// The two calls that a decoding step makes for every layer, append_kv8 and attention_kv8, straight from
// torch tensors to the library's C entry points: the checks, the output's allocation and the current
// stream, which in Python took longer than such a step's kernels run.  The entry points come as
// addresses from the library that the package loaded, so this file links to none.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "qkq.h"

namespace {

decltype(&qkq_append_kv8) append_kv8;
decltype(&qkq_attention_kv8) attention_kv8;
decltype(&qkq_attention_kv8_workspace_bytes) workspace_bytes;

// A refused argument: a ValueError.
void need(bool ok, const char *what) { TORCH_CHECK_VALUE(ok, what); }

const at::Tensor *optional(PyObject *o, const char *name)
{
    if (o == Py_None) return nullptr;
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return &THPVariable_Unpack(o);
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

template <typename T>
T *address(const at::Tensor *t)
{
    return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}

bool like(const at::Tensor &t, at::IntArrayRef shape, at::ScalarType type, const at::Device &dev)
{
    return t.sizes() == shape && t.scalar_type() == type && t.is_contiguous() && t.device() == dev;
}

int dtype_of(const at::Tensor &t, const char *what)
{
    need(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf, what);
    return t.scalar_type() == at::kBFloat16 ? QKQ_DTYPE_BF16 : QKQ_DTYPE_FP16;
}

// The cache and the index tensors of a call.
struct Cache {
    const at::Tensor &k, &v, &ks, &vs, &table, &lens;
    const at::Tensor *cu;
    int64_t pages, Hkv, page, d, B, max_pages;

    Cache(PyObject *const *a, const at::Device &dev, int64_t T)
        : k(tensor(a[0], "cache.k")), v(tensor(a[1], "cache.v")), ks(tensor(a[2], "cache.k_steps")), vs(tensor(a[3], "cache.v_steps")),
          table(tensor(a[4], "block_table")), lens(tensor(a[5], "seq_lens")), cu(optional(a[6], "cu_new"))
    {
        need(dev.is_cuda(), "tensors must be on a CUDA device");
        need(k.scalar_type() == at::kFloat8_e4m3fn && v.scalar_type() == at::kFloat8_e4m3fn, "cache codes must be float8_e4m3fn");
        need(ks.scalar_type() == at::kFloat && vs.scalar_type() == at::kFloat, "cache steps must be float32");
        need(k.dim() == 4 && v.sizes() == k.sizes() && ks.sizes() == k.sizes().slice(0, 2) && vs.sizes() == ks.sizes(),
             "cache shapes differ: codes [pages, Hkv, page_size, d_h], steps [pages, Hkv]");
        pages = k.size(0);
        Hkv = k.size(1);
        page = k.size(2);
        d = k.size(3);
        need(table.dim() == 2 && lens.dim() == 1 && lens.size(0) == table.size(0), "block_table must be [B, max_pages] and seq_lens [B]");
        B = table.size(0);
        max_pages = table.size(1);
        if (cu)
            need(cu->dim() == 1 && cu->size(0) == B + 1, "cu_new must be [B + 1]");
        else
            need(T == B, "without cu_new there is one new token per sequence");
        need(table.scalar_type() == at::kInt && lens.scalar_type() == at::kInt && (!cu || cu->scalar_type() == at::kInt),
             "block_table, seq_lens and cu_new must be int32");
        for (const at::Tensor *t : {&k, &v, &ks, &vs, &table, &lens, cu}) {
            if (!t) continue;
            need(t->is_contiguous(), "the cache and the index tensors must be contiguous");
            need(t->device() == dev, "all tensors must be on one CUDA device");
        }
        // the C entry points take these as int
        need(B < INT32_MAX && max_pages <= INT32_MAX && Hkv <= INT32_MAX && page <= INT32_MAX && d <= INT32_MAX, "sizes beyond 32 bits");
    }
};

// Elements from token to token of [T, heads, d] rows, each token's heads contiguous.
int64_t row_stride(const at::Tensor &t, const char *name, int64_t T, int64_t H, const Cache &c, at::ScalarType type, const at::Device &dev)
{
    const int64_t shape[3] = {T, H, c.d};
    TORCH_CHECK_VALUE(t.sizes() == at::IntArrayRef(shape, 3) && t.scalar_type() == type && t.device() == dev, name,
                      " must be [T, heads, d_h] of one type and device with the others");
    const auto s = t.strides();
    if (t.numel())
        TORCH_CHECK_VALUE(s[2] == 1 && (H == 1 || s[1] == c.d), name, ": the heads of a token must be contiguous");
    return T > 1 ? s[0] : std::max(s[0], H * c.d) / 8 * 8;
}

const at::Tensor *status_of(PyObject *o, const at::Device &dev)
{
    const at::Tensor *t = optional(o, "status");
    need(!t || (t->scalar_type() == at::kInt && t->numel() > 0 && t->device() == dev), "status must be int32 on the tensors' device");
    return t;
}

// The stream's handle: the one given, or the device's current one.
qkq_stream_t stream_of(PyObject *o, const at::Device &dev)
{
    if (o == Py_None) return reinterpret_cast<qkq_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
    void *p = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw python_error();
    return reinterpret_cast<qkq_stream_t>(p);
}

int64_t integer(PyObject *o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

// append(k, v, cache (4), block_table, seq_lens, cu_new, q, pos, cos, sin, style, q_out, status, stream)
// -> (code, q_out)
PyObject *py_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 17 && append_kv8, "append takes 17 arguments");
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    need(k.dim() == 3, "k must be [T, heads, d_h]");
    const at::Device dev = k.device();
    const at::ScalarType type = k.scalar_type();
    const int dtype = dtype_of(k, "k must be bfloat16 or float16");
    const int64_t T = k.size(0);
    const Cache c(a + 2, dev, T);
    const int64_t k_stride = row_stride(k, "k", T, c.Hkv, c, type, dev), v_stride = row_stride(v, "v", T, c.Hkv, c, type, dev);
    const at::Tensor *q = optional(a[9], "q"), *pos = optional(a[10], "pos"), *cos = optional(a[11], "cos_tab"), *sin = optional(a[12], "sin_tab");
    const at::Tensor *q_out = optional(a[14], "q_out"), *status = status_of(a[15], dev);
    const c10::cuda::CUDAGuard guard(dev);
    int64_t Hq = c.Hkv, q_stride = 0;
    at::Tensor made;
    if (q) {
        need(q->dim() == 3, "q must be [T, heads, d_h]");
        Hq = q->size(1);
        need(Hq <= INT32_MAX, "sizes beyond 32 bits");
        q_stride = row_stride(*q, "q", T, Hq, c, type, dev);
        if (!q_out) {
            made = at::empty({T, Hq, c.d}, q->options().memory_format(at::MemoryFormat::Contiguous));
            q_out = &made;
        } else {
            need(like(*q_out, q->sizes(), type, dev), "q_out must be a contiguous tensor like q");
        }
    } else {
        need(!q_out, "q_out without q");
    }
    need(!cos == !sin, "cos_tab and sin_tab go together");
    int64_t max_pos = 0, rot = 0;
    if (cos) {
        need(cos->dim() == 2 && like(*cos, cos->sizes(), at::kFloat, dev) && like(*sin, cos->sizes(), at::kFloat, dev),
             "cos_tab and sin_tab must be contiguous float32 [max_pos, rot_dim/2]");
        max_pos = cos->size(0);
        rot = 2 * cos->size(1);
        need(max_pos <= INT32_MAX && rot <= INT32_MAX, "sizes beyond 32 bits");
    }
    need(!pos || like(*pos, {T}, at::kInt, dev), "pos must be int32 [T]");
    const int style = static_cast<int>(integer(a[13]));
    const qkq_stream_t s = stream_of(a[16], dev);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = append_kv8(address<void>(q), q_stride, k.data_ptr(), k_stride, v.data_ptr(), v_stride, dtype, address<int32_t>(pos), T, address<int32_t>(c.cu),
                    address<int32_t>(&c.lens), static_cast<int>(c.B), address<int32_t>(&c.table), static_cast<int>(c.max_pages), c.pages,
                    static_cast<int>(c.page), static_cast<int>(Hq), static_cast<int>(c.Hkv), static_cast<int>(c.d), static_cast<int>(rot), style,
                    address<float>(cos), address<float>(sin), static_cast<int>(max_pos), address<void>(q_out), address<uint8_t>(&c.k),
                    address<uint8_t>(&c.v), address<float>(&c.ks), address<float>(&c.vs), address<int>(status), s);
    Py_END_ALLOW_THREADS
    PyObject *out = made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[14]);
    if (!out) throw python_error();
    return Py_BuildValue("(iN)", rc, out);
    END_HANDLE_TH_ERRORS
}

// attention(q, cache (4), block_table, seq_lens, cu_new, scale, window, sinks, out, lse, workspace, status, stream)
// -> (code, out)
PyObject *py_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 16 && attention_kv8, "attention takes 16 arguments");
    const at::Tensor &q = tensor(a[0], "q");
    need(q.dim() == 3, "q must be [T, heads, d_h]");
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const int dtype = dtype_of(q, "q must be bfloat16 or float16");
    const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2);
    const Cache c(a + 1, dev, T);
    need(d == c.d && q.is_contiguous(), "q must be contiguous [T, Hq, d_h] with the cache's d_h");
    need(Hq <= INT32_MAX, "sizes beyond 32 bits");
    const at::Tensor *out = optional(a[11], "out"), *lse = optional(a[12], "lse"), *ws = optional(a[13], "workspace"), *status = status_of(a[14], dev);
    float scale;
    if (a[8] == Py_None) {
        scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    } else {
        scale = static_cast<float>(PyFloat_AsDouble(a[8]));
        if (PyErr_Occurred()) throw python_error();
    }
    const int64_t window = integer(a[9]), sinks = integer(a[10]);
    need(window <= INT32_MAX && window >= INT32_MIN && sinks <= INT32_MAX && sinks >= INT32_MIN, "window and sinks must be 32-bit integers");
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor made, space;
    if (!out) {
        made = at::empty(q.sizes(), q.options().memory_format(at::MemoryFormat::Contiguous));
        out = &made;
    } else {
        need(like(*out, q.sizes(), type, dev), "out must be a contiguous tensor like q");
    }
    need(!lse || like(*lse, {T, Hq}, at::kFloat, dev), "lse must be contiguous float32 [T, Hq]");
    size_t size;
    if (ws) {
        need(ws->device() == dev && ws->is_contiguous(), "workspace must be contiguous on the tensors' device");
        size = ws->nbytes();
    } else {
        size = workspace_bytes(T, static_cast<int>(c.B), static_cast<int>(Hq), static_cast<int>(c.Hkv), static_cast<int>(d));
        if (size) {
            space = at::empty({static_cast<int64_t>(size)}, q.options().dtype(at::kByte));
            ws = &space;
        }
    }
    const qkq_stream_t s = stream_of(a[15], dev);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = attention_kv8(q.data_ptr(), dtype, T, address<int32_t>(c.cu), address<int32_t>(&c.lens), static_cast<int>(c.B), address<int32_t>(&c.table),
                       static_cast<int>(c.max_pages), c.pages, static_cast<int>(c.page), address<uint8_t>(&c.k), address<uint8_t>(&c.v),
                       address<float>(&c.ks), address<float>(&c.vs), static_cast<int>(Hq), static_cast<int>(c.Hkv), static_cast<int>(d), scale,
                       static_cast<int>(window), static_cast<int>(sinks), out->data_ptr(), address<float>(lse), address<void>(ws), size,
                       address<int>(status), s);
    Py_END_ALLOW_THREADS
    PyObject *o = made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[11]);
    if (!o) throw python_error();
    return Py_BuildValue("(iN)", rc, o);
    END_HANDLE_TH_ERRORS
}

// init(append, attention, workspace_bytes): the entry points' addresses
PyObject *py_init(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 3, "init takes 3 addresses");
    append_kv8 = reinterpret_cast<decltype(append_kv8)>(integer(a[0]));
    attention_kv8 = reinterpret_cast<decltype(attention_kv8)>(integer(a[1]));
    workspace_bytes = reinterpret_cast<decltype(workspace_bytes)>(integer(a[2]));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_append)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_attention)), METH_FASTCALL, nullptr},
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_init)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "qkq_binding", nullptr, -1, methods};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit_qkq_binding() { return PyModule_Create(&module); }
