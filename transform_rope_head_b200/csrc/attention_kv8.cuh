// What the kernels of the attention over the paged 8-bit cache share: the work line and how a CTA
// finds its part of it, the partial rows that parts of a unit leave, and the output rows.
#pragma once

#include <math.h>

#include <atomic>

#include "kv8.cuh"

namespace qkq {

constexpr int KV8_MAX_CTAS = 512;  // above the persistent grids here (148 SMs x 3)

// Where a CTA's part begins: with tile j0 of (b, qt, hk), the unit at place u0 of the line (j0 = 0 where the
// part is empty).
struct KV8Meta {
    int64_t u0;
    int j0, b, qt, hk;
};

// The workspace: per CTA its beginning, and two partial units (its first, and its last where that is
// another one), each R rows of unnormalised outputs with (maximum, sum).
struct KV8Partials {
    KV8Meta *meta;
    float *ml, *o;
    static constexpr size_t META = 32;
    __host__ __device__ KV8Partials(void *ws, int ctas, int rows, int d_h)
    {
        char *c = static_cast<char *>(ws);
        meta = reinterpret_cast<KV8Meta *>(c);
        ml = reinterpret_cast<float *>(c + META * ctas);
        o = ml + static_cast<size_t>(ctas) * 2 * rows * 2;
    }
    static size_t bytes(int ctas, int rows, int d_h)
    {
        return ctas * (META + static_cast<size_t>(2) * rows * (2 + d_h) * sizeof(float));
    }
};
static_assert(sizeof(KV8Meta) <= KV8Partials::META, "workspace layout");

// A sequence whose rows lie outside the buffers has none; one whose length does has no cached
// tokens (its rows come out empty).
__device__ __forceinline__ KV8Seq kv8_seq_checked(const KV8Index &x, int b)
{
    KV8Seq s = kv8_seq(x, b);
    if (!s.ok) {
        const bool rows = s.q0 >= 0 && s.n >= 0 && static_cast<int64_t>(s.q0) + s.n <= x.T;
        if (!rows) s.n = 0;
        s.len = 0;
    }
    return s;
}

// Tiles of TS cached tokens that some row of a unit (rows qt * R ..) sees: tile j of the unit is
// tile j of the sequence for j < head, j + skip after.
struct KV8Span {
    int count, head, skip;
    int first, last;  // index in the sequence of the first and last row's token
};

template <int TS>
__device__ __forceinline__ KV8Span unit_span(const AttnKV8Params &p, const KV8Seq &s, int qt, int R)
{
    KV8Span u;
    const int r0 = qt * R, r1 = min(r0 + R, s.n * p.ratio) - 1;
    u.first = s.len - s.n + p.div_ratio(r0);
    u.last = s.len - s.n + p.div_ratio(r1);
    const int end = max(u.last + 1, 0);  // <= len
    const int lo = p.window > 0 ? max(u.first - p.window + 1, 0) : 0;
    const int sink = p.window > 0 ? (min(p.sinks, end) + TS - 1) / TS : 0;
    const int w0 = min(lo, end) / TS, w1 = (end + TS - 1) / TS;
    if (w0 > sink) {
        u.head = sink;
        u.skip = w0 - sink;
        u.count = sink + w1 - w0;
    } else {
        u.head = w1;
        u.skip = 0;
        u.count = w1;
    }
    u.count = max(u.count, 1);  // a unit without tokens still writes its rows
    return u;
}

__device__ __forceinline__ int unit_blocks(const AttnKV8Params &p, const KV8Seq &s, int R)
{
    return (s.n * p.ratio + R - 1) / R;
}

// Places of a sequence on the line over all its query blocks and key heads; each lane of the warp asks for
// its own (b < 0: none).  Long lists of blocks are summed by the whole warp.  one: the places of a unit
// where the sequence has one query block, else 0.
template <int TS>
__device__ __forceinline__ int64_t seq_places(const AttnKV8Params &p, int b, int R, int extra, int lane, int &one, int &bad)
{
    int64_t w = 0;
    int blocks = 0;
    one = 0;
    if (b >= 0) {
        bad |= !kv8_seq(p.x, b).ok;
        const KV8Seq s = kv8_seq_checked(p.x, b);
        blocks = unit_blocks(p, s, R);
        if (blocks == 1) w = one = unit_span<TS>(p, s, 0, R).count + extra;
    }
    for (unsigned m = __ballot_sync(FULL_MASK, blocks > 1); m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const KV8Seq s = kv8_seq_checked(p.x, __shfl_sync(FULL_MASK, b, src));
        const int n = __shfl_sync(FULL_MASK, blocks, src);
        int64_t sum = 0;
        for (int q = lane; q < n; q += 32) sum += unit_span<TS>(p, s, q, R).count + extra;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
        if (lane == src) w = sum;
    }
    return w * p.Hkv;
}

struct KV8Start {
    int64_t lo, hi, base, u0;
    int b, qt, hk, j0, flags;
    int found;  // qt, hk, j0 and u0 are in place without the search by warp 0
    int64_t warp_sum[2][32];
};

// Place lo of a unit's c places per key head, r places after the first head's first.
__device__ __forceinline__ void start_at(KV8Start &st, int64_t lo, int64_t r, int c, int extra, bool small)
{
    const int64_t h = small ? static_cast<uint32_t>(r) / static_cast<uint32_t>(c) : r / c;
    const int at = static_cast<int>(r - h * c);
    st.hk = static_cast<int>(h);
    st.j0 = max(at - extra, 0);
    st.u0 = lo - at;
}

// The CTA's part [lo, hi) of the line of all tiles (sequence, query block, key head, tile), on which a unit has
// `extra` places before its tiles' (what beginning and ending it costs, in tiles), and the unit that holds lo:
// it begins at place u0, the part with its tile j0.  Every thread of the CTA calls it.  least: places a part
// has at least.
template <int TS, int R, int THREADS>
__device__ __forceinline__ void find_start(const AttnKV8Params &p, KV8Start &st, int extra, int least)
{
    constexpr int NWARP = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int B = p.x.B;
    int64_t sum = 0, mine = 0;
    int bad = 0, one = 0;
    for (int b0 = 0; b0 < B; b0 += THREADS) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        mine = seq_places<TS>(p, b < B ? b : -1, R, extra, lane, one, bad);
        sum += mine;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(FULL_MASK, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) st.warp_sum[0][warp] = sum;
    bad = __syncthreads_or(bad);
    int64_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < NWARP; ++w) {
        if (w == warp) before = total;
        total += st.warp_sum[0][w];
    }
    // 64-bit divisions are long, and hardly a line needs them
    const bool small = total < 0x7fffffff;
    const int64_t share = small ? (static_cast<uint32_t>(total) + gridDim.x - 1) / gridDim.x : (total + gridDim.x - 1) / gridDim.x;
    const int64_t len = share < least ? least : share;
    const int64_t lo = min(len * blockIdx.x, total), hi = min(lo + len, total);
    if (threadIdx.x == 0) {
        st.lo = lo;
        st.hi = hi;
        st.flags = bad ? ST_CACHE_INDEX : 0;
    }
    if (lo >= hi) {
        if (threadIdx.x == 0) {
            st.b = st.qt = st.hk = st.j0 = 0;
            st.u0 = lo;
        }
        __syncthreads();
        return;
    }
    if (B <= THREADS) {
        // a sequence a thread: the one that holds lo says where
        sum += before;
        if (lo >= sum - mine && lo < sum) {
            st.b = threadIdx.x;
            st.base = sum - mine;
            st.qt = 0;
            st.found = one > 0;
            if (one) start_at(st, lo, lo - (sum - mine), one, extra, small);
        }
        __syncthreads();
    } else {
        int64_t base = 0;
        if (threadIdx.x == 0) st.found = 0;
        for (int b0 = 0; b0 < B; b0 += THREADS) {
            const int b = b0 + static_cast<int>(threadIdx.x);
            const int64_t w = seq_places<TS>(p, b < B ? b : -1, R, extra, lane, one, bad);
            int64_t inc = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(FULL_MASK, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) st.warp_sum[1][warp] = inc;
            __syncthreads();
            int64_t first = base;
#pragma unroll
            for (int k = 0; k < NWARP; ++k) {
                if (k < warp) first += st.warp_sum[1][k];
                base += st.warp_sum[1][k];
            }
            inc += first;
            if (b < B && lo >= inc - w && lo < inc) {
                st.b = b;
                st.base = inc - w;
            }
            __syncthreads();
            if (lo < base) break;
        }
    }
    // Written before the last barrier above and not again: every warp takes the same way here, however late
    // it reads, and so the same barriers (the search below must not set it).
    if (st.found) return;
    if (warp == 0) {
        const KV8Seq s = kv8_seq_checked(p.x, st.b);
        const int blocks = unit_blocks(p, s, R);
        int64_t rem = lo - st.base;
        for (int q0 = 0; q0 < blocks; q0 += 32) {
            const int q = q0 + lane;
            const int c = q < blocks ? unit_span<TS>(p, s, q, R).count + extra : 0;
            const int64_t w = static_cast<int64_t>(c) * p.Hkv;
            int64_t inc = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(FULL_MASK, inc, o);
                if (lane >= o) inc += y;
            }
            if (rem >= inc - w && rem < inc) {
                st.qt = q;
                start_at(st, lo, rem - (inc - w), c, extra, small);
            }
            const int64_t all = __shfl_sync(FULL_MASK, inc, 31);
            if (rem < all) break;
            rem -= all;
        }
    }
    __syncthreads();
}

// The unit after (b, qt, hk); there is one.
__device__ __forceinline__ void next_unit(const AttnKV8Params &p, const KV8Seq &s, int R, int &b, int &qt, int &hk)
{
    if (++hk < p.Hkv) return;
    hk = 0;
    if (++qt < unit_blocks(p, s, R)) return;
    qt = 0;
    do {
        ++b;
    } while (b < p.x.B - 1 && kv8_seq_checked(p.x, b).n == 0);
}

// The weights 2^(logit - m) are rounded to fp16 for their product with the values.  A row's m stands KV8_UP below
// its largest logit when it moves, and moves when a logit passes that one by KV8_SLACK, so that rescaling is
// rare: a weight is at most 2^(KV8_UP + KV8_SLACK) = 2^15, which fp16 holds, and what its subnormals
// round off is 2^-(25 + KV8_UP) of the largest weight or less.  (With the largest logit itself as m, rows
// that a first token of no value dominates by 2^25 were 7% off.)
constexpr float KV8_SLACK = 8.0f, KV8_UP = 7.0f;

// Two weights as fp16, to nearest.  Saturating: beyond logits of 2^24 the offset's own fp32 rounding can let a weight
// pass 2^15, and an infinite one would make the row NaN.
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 2^e of a row's scaling into fp16: the row's largest magnitude goes to [2^14, 2^15), so that
// what fp16 flushes is 2^-38 of it.
__device__ __forceinline__ int row_exponent(float amax)
{
    const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14;
    return amax > 0.0f ? max(e, -126) : 0;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// N channels of row rr of (sequence s, key head hk): the normalised output (0 where the row saw
// nothing), and with the first ones the row's log-sum-exp.
template <int N>
__device__ __forceinline__ void store_row(const AttnKV8Params &p, const KV8Seq &s, int rr, int hk, int c, int d_h,
                                          const float (&acc)[N], float top, float sum)
{
    const int token = p.div_ratio(rr);
    const int64_t row = static_cast<int64_t>(s.q0) * p.Hq + hk * p.ratio + rr + static_cast<int64_t>(token) * (p.Hq - p.ratio);
    const bool empty = top == -INFINITY && sum == 0.0f;
    const float inv = empty ? 0.0f : 1.0f / sum;
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = empty ? 0u : pack16(acc[2 * i] * inv, acc[2 * i + 1] * inv, p.half);
    uint16_t *dst = p.out + row * d_h + c;
    if (N == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[N / 2 - 1]);
    else
        *reinterpret_cast<uint32_t *>(dst) = w[0];
    if (c == 0 && p.lse) p.lse[row] = empty ? -INFINITY : (lg2(sum) + top) * 0.6931471805599453f;
}

// Query rows a unit of the tensor-memory kernel has, and whether a call takes that kernel: from more than 24
// rows a sequence on, what the register kernel takes in one unit (16 sequences of 8000 tokens, d_h 128: 24
// rows 101 us against 126, 32 rows 186 against 126; d_h 64: 73 against 101, 141 against 101).
constexpr int KV8_TC_ROWS = 256, KV8_TC_MAX_CTAS = 160;
inline bool kv8_takes_tc(int64_t T, int B, int ratio) { return T * ratio > static_cast<int64_t>(B) * 24; }
// Allows a kernel its dynamic shared memory, once per device (the call costs more than a launch's arguments).
// done: a bit per device ordinal, the kernel's own.
template <typename Kernel>
cudaError_t allow_smem(std::atomic<uint64_t> &done, Kernel kern, int bytes, int ordinal)
{
    const uint64_t bit = ordinal < 64 ? 1ull << ordinal : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

cudaError_t attention_kv8_tc_launch(const AttnKV8Params &p, int d_h, const DeviceInfo &dev, cudaStream_t stream);
// Joins the partial rows that `ctas` CTAs left, R rows a unit.
cudaError_t attention_kv8_join_launch(const AttnKV8Params &p, int d_h, int ctas, int R, cudaStream_t stream);

}  // namespace qkq
