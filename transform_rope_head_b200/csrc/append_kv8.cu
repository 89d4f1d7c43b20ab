// Appending keys and values to the paged 8-bit cache, RoPE on the way; queries rotated in the
// same launch.
//
// Per page and key head: y = RoPE(k) on the first rot channels (fp32, a' = fma(a, c, -(b*s)),
// b' = fma(a, s, b*c)), the rest as they are; step s = 2^ceil(log2(max|y| / 448)) over the
// page's new tokens, at least the page's present step where it was partly full; code =
// e4m3(y / s), one rounding (1/s is exact).  Where a partly full page's step grows, the rows it
// holds are rounded again to the new step: a power of two apart, so only values that fall
// under e4m3's smallest normal change.
//
// Memory bound: 2 bytes in per key, value and query channel, 1 byte out per key and value
// channel, 2 per query channel.  One warp owns 16 rows of one page and head (K or V), all
// their loads in flight at once, the values in registers between the maximum and the
// quantiser, so the input is read once; pages of more than 16 tokens take several warps,
// which share the maximum through shared memory.  A lane owns 16 channels of a row: the two
// 8-channel chunks whose pairs rotate together, so RoPE needs no exchange.  A query warp owns
// one token and 16 heads and keeps the token's cos / sin in registers for all of them.
#include "kv8.cuh"

namespace qkq {

namespace {

constexpr int AK_WARPS = 8;
constexpr int AK_QHEADS = 16;  // query heads per warp

// The pair table of a lane: 8 pairs' cos and sin.
struct Turn {
    float c[8], s[8];
};

__device__ __forceinline__ void load_turn(Turn &r, const AppendKV8Params &p, int m, int q, int &flags)
{
    const int64_t row = clamp_pos(m, p.max_pos, flags);
    const float4 *c = reinterpret_cast<const float4 *>(p.cos_t + row * (p.rot / 2) + 8 * q);
    const float4 *s = reinterpret_cast<const float4 *>(p.sin_t + row * (p.rot / 2) + 8 * q);
    const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
    r.c[0] = c0.x, r.c[1] = c0.y, r.c[2] = c0.z, r.c[3] = c0.w;
    r.c[4] = c1.x, r.c[5] = c1.y, r.c[6] = c1.z, r.c[7] = c1.w;
    r.s[0] = s0.x, r.s[1] = s0.y, r.s[2] = s0.z, r.s[3] = s0.w;
    r.s[4] = s1.x, r.s[5] = s1.y, r.s[6] = s1.z, r.s[7] = s1.w;
}

__device__ __forceinline__ void turn_pair(float &a, float &b, float c, float s)
{
    const float x = __fmaf_rn(a, c, -__fmul_rn(b, s));
    b = __fmaf_rn(a, s, __fmul_rn(b, c));
    a = x;
}

// y[0..7] = first chunk, y[8..15] = second.
__device__ __forceinline__ void turn16(float (&y)[16], const Turn &r, bool interleaved)
{
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_pair(y[2 * e], y[2 * e + 1], r.c[e], r.s[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_pair(y[e], y[e + 8], r.c[e], r.s[e]);
    }
}

// Chunk pair q of a row: its two 8-channel chunks.  Half layout: chunk q pairs with q + rot/16
// below rot; elsewhere (and interleaved) neighbours.
__device__ __forceinline__ void chunks_of(int q, const AppendKV8Params &p, int &c0, int &c1)
{
    const bool apart = !p.interleaved && q < p.rot / 16;
    c0 = apart ? q : 2 * q;
    c1 = apart ? q + p.rot / 16 : 2 * q + 1;
}

__device__ __forceinline__ void unpack8(float *y, const uint4 &w, bool half)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 v = unpack16(u[e], half);
        y[2 * e] = v.x;
        y[2 * e + 1] = v.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float *y, bool half)
{
    return make_uint4(pack16(y[0], y[1], half), pack16(y[2], y[3], half), pack16(y[4], y[5], half),
                      pack16(y[6], y[7], half));
}

// e4m3 of 8 values times inv, saturating (NaN stays NaN).
__device__ __forceinline__ uint2 quant8(const float *y, float inv)
{
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(__fmul_rn(y[4 * h], inv), __fmul_rn(y[4 * h + 1], inv)), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(__fmul_rn(y[4 * h + 2], inv), __fmul_rn(y[4 * h + 3], inv)), __NV_SATFINITE, __NV_E4M3);
        w[h] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint2 requant8(uint2 w, float ratio)
{
    float y[8];
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t a = e4m3x2_to_half2(u[h] & 0xffffu), b = e4m3x2_to_half2(u[h] >> 16);
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&b));
        y[4 * h] = x.x, y[4 * h + 1] = x.y, y[4 * h + 2] = z.x, y[4 * h + 3] = z.y;
    }
    return quant8(y, ratio);
}

// The smallest 2^e with amax <= 448 * 2^e, e clamped to +-40 (448 = 1.75 * 2^8; amax = 0: 2^-40).
__device__ __forceinline__ float step_of(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = min(max(e, -40), 40);
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// DH channels; WPU warps (16 rows each) per page and head.  BLOCKS on an SM: 3 for many tokens, where a few
// spilled registers cost less than loads in flight gain (8 prompts of 4096: 153 us against 160), 2
// for a token a sequence (256 sequences: 7.7 us against 7.9).
template <int DH, int WPU, int BLOCKS>
__global__ void __launch_bounds__(AK_WARPS * 32, BLOCKS)
k_append_kv8(const AppendKV8Params p)
{
    constexpr int NQ = DH / 16;        // lanes per row
    constexpr int RPI = 32 / NQ;       // rows per iteration
    constexpr int IT = 16 / RPI;       // iterations over a warp's 16 rows
    __shared__ float s_amax[AK_WARPS];
    wait_prior_grid();
    allow_next_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int q = lane % NQ, rl = lane / NQ;
    const KV8Index &x = p.x;
    const bool half = p.half;
    int flags = 0;
    int c0, c1;
    chunks_of(q, p, c0, c1);
    const bool turns = q < p.rot / 16;

    if (blockIdx.x >= p.kv_ctas) {
        // queries: one token, 16 heads
        const int64_t unit = static_cast<int64_t>(blockIdx.x - p.kv_ctas) * AK_WARPS + warp;
        const int blocks = (p.Hq + AK_QHEADS - 1) / AK_QHEADS;
        const int64_t t = unit / blocks;
        const int h0 = static_cast<int>(unit % blocks) * AK_QHEADS;
        bool live = t < x.T;
        int m = 0;
        if (live) {
            const int B = x.B;
            const int last = x.cu ? __ldg(x.cu + B) : B;
            live = t < last;
            if (live && p.pos) {
                m = __ldg(p.pos + t);
            } else if (live) {
                int b = static_cast<int>(t);
                if (x.cu) b = warp_upper(B, t, lane, [&](int i) { return static_cast<int64_t>(__ldg(x.cu + i)); });
                const KV8Seq s = kv8_seq(x, b);
                // a row of no sequence (rows before the first) stays as it is
                live = t >= s.q0 && t < static_cast<int64_t>(s.q0) + s.n;
                m = s.len - s.n + static_cast<int>(t - s.q0);
            }
        }
        if (!live) return;
        Turn r;
        if (turns) load_turn(r, p, m, q, flags);
        constexpr int HI = AK_QHEADS / RPI;
        uint4 a[HI], b[HI];
#pragma unroll
        for (int i = 0; i < HI; ++i) {
            const int h = h0 + i * RPI + rl;
            if (h < p.Hq) {
                const uint16_t *src = p.q + t * p.q_stride + h * DH;
                a[i] = __ldg(reinterpret_cast<const uint4 *>(src + 8 * c0));
                b[i] = __ldg(reinterpret_cast<const uint4 *>(src + 8 * c1));
            }
        }
#pragma unroll
        for (int i = 0; i < HI; ++i) {
            const int h = h0 + i * RPI + rl;
            if (h < p.Hq) {
                uint16_t *dst = p.q_out + (t * p.Hq + h) * DH;
                if (turns) {
                    float y[16];
                    unpack8(y, a[i], half);
                    unpack8(y + 8, b[i], half);
                    turn16(y, r, p.interleaved);
                    a[i] = pack8(y, half);
                    b[i] = pack8(y + 8, half);
                }
                *reinterpret_cast<uint4 *>(dst + 8 * c0) = a[i];
                *reinterpret_cast<uint4 *>(dst + 8 * c1) = b[i];
            }
        }
        if (flags && p.status) atomicOr(p.status, flags);
        return;
    }

    // keys and values: unit = (page slot, K or V, head), WPU warps each
    constexpr int UNITS = AK_WARPS / WPU;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * UNITS + warp / WPU;
    const int w_in = warp % WPU;
    const int64_t slot = unit / (2 * p.Hkv);
    const int kvh = static_cast<int>(unit % (2 * p.Hkv));
    const bool is_v = kvh >= p.Hkv;
    const int h = is_v ? kvh - p.Hkv : kvh;
    bool live = slot < p.slots;
    KV8Seq s{};
    int b = 0, pi = 0, before = 0, page = -1;
    if (live) {
        if (x.cu) {
            // sequence b owns the page slots from cu[b] / page + 2 b on: at least as many as the
            // pages its new tokens can touch
            b = warp_upper(x.B, slot, lane, [&](int i) {
                return static_cast<int64_t>(__ldg(x.cu + i) >> x.page_shift) + 2 * i;
            });
            s = kv8_seq(x, b);
            before = s.len - s.n;
            live = s.ok && before >= 0;
            if (!live) flags |= ST_CACHE_INDEX;
            const int64_t off = slot - ((s.q0 >> x.page_shift) + 2 * static_cast<int64_t>(b));
            pi = (before >> x.page_shift) + static_cast<int>(off);
            live = live && off >= 0 && s.n > 0 && pi <= (s.len - 1) >> x.page_shift;
        } else {
            b = static_cast<int>(slot);
            s = kv8_seq(x, b);
            before = s.len - 1;
            live = s.ok && before >= 0;
            if (!live) flags |= ST_CACHE_INDEX;
            pi = live ? before >> x.page_shift : 0;
        }
    }
    if (live) {
        page = kv8_page(x, b, pi);
        if (page < 0) {
            flags |= ST_CACHE_INDEX;
            live = false;
        }
    }
    const int64_t ph = static_cast<int64_t>(page) * p.Hkv + h;
    float *const steps = is_v ? p.v_steps : p.k_steps;
    uint8_t *const codes = (is_v ? p.v_codes : p.k_codes) + (live ? (ph << x.page_shift) * DH : 0);
    const int first = pi << x.page_shift;  // index in the sequence of the page's row 0
    const int held = live ? max(0, before - first) : 0;
    float amax = 0.0f, old = 0.0f;
    float y[IT][16];
    if (live) {
        if (held > 0) old = steps[ph];
        const uint16_t *src = is_v ? p.v : p.k;
        const int64_t stride = is_v ? p.v_stride : p.k_stride;
        uint4 a[IT], c[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int at = first + w_in * 16 + i * RPI + rl;
            a[i] = c[i] = make_uint4(0, 0, 0, 0);
            if (at >= before && at < s.len) {
                const uint16_t *row = src + static_cast<int64_t>(s.q0 + at - before) * stride + h * DH;
                a[i] = __ldg(reinterpret_cast<const uint4 *>(row + 8 * c0));
                c[i] = __ldg(reinterpret_cast<const uint4 *>(row + 8 * c1));
            }
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int at = first + w_in * 16 + i * RPI + rl;
            unpack8(y[i], a[i], half);
            unpack8(y[i] + 8, c[i], half);
            if (!is_v && turns && at >= before && at < s.len) {
                Turn r;
                load_turn(r, p, p.pos ? __ldg(p.pos + s.q0 + at - before) : at, q, flags);
                turn16(y[i], r, p.interleaved);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float v = fabsf(y[i][e]);
                if (v <= 3.402823466e38f)
                    amax = fmaxf(amax, v);
                else
                    flags |= ST_NONFINITE;
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, o));
    }
    if (WPU > 1) {
        if (lane == 0) s_amax[warp] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WPU; ++i) amax = fmaxf(amax, s_amax[warp / WPU * WPU + i]);
    }
    if (live) {
        const float step = fmaxf(step_of(amax), old);
        if (amax > 448.0f * step) flags |= ST_SCALE_OVERFLOW;
        const float inv = __fdiv_rn(1.0f, step);
        const float ratio = old < step ? old / step : 1.0f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int row = w_in * 16 + i * RPI + rl;
            const int at = first + row;
            uint8_t *dst = codes + row * DH;
            if (at >= before && at < s.len) {
                *reinterpret_cast<uint2 *>(dst + 8 * c0) = quant8(y[i], inv);
                *reinterpret_cast<uint2 *>(dst + 8 * c1) = quant8(y[i] + 8, inv);
            } else if (row < held && ratio < 1.0f) {
                uint2 *u = reinterpret_cast<uint2 *>(dst + 8 * c0), *v = reinterpret_cast<uint2 *>(dst + 8 * c1);
                *u = requant8(*u, ratio);
                *v = requant8(*v, ratio);
            }
        }
        if (w_in == 0 && lane == 0) steps[ph] = step;
    }
    if (p.status) {
        flags = __reduce_or_sync(FULL_MASK, flags);
        if (flags && lane == 0) atomicOr(p.status, flags);
    }
}

template <int DH, int BLOCKS>
cudaError_t launch(const AppendKV8Params &p, int64_t ctas, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(ctas)), block(AK_WARPS * 32);
    switch (p.x.page_shift) {
        case 4: return launch_after_prior(k_append_kv8<DH, 1, BLOCKS>, grid, block, 0, stream, p);
        case 5: return launch_after_prior(k_append_kv8<DH, 2, BLOCKS>, grid, block, 0, stream, p);
        case 6: return launch_after_prior(k_append_kv8<DH, 4, BLOCKS>, grid, block, 0, stream, p);
        default: return launch_after_prior(k_append_kv8<DH, 8, BLOCKS>, grid, block, 0, stream, p);
    }
}

}  // namespace

cudaError_t append_kv8_launch(AppendKV8Params p, int d_h, cudaStream_t stream)
{
    // page slots: one per sequence when each has one new token, else as counted in the kernel
    p.slots = p.x.cu ? (p.x.T >> p.x.page_shift) + 2 * static_cast<int64_t>(p.x.B) : p.x.B;
    const int units = AK_WARPS >> (p.x.page_shift - 4);
    const int64_t kv = (p.slots * 2 * p.Hkv + units - 1) / units;
    const int64_t qw = p.q ? p.x.T * ((p.Hq + AK_QHEADS - 1) / AK_QHEADS) : 0;
    const int64_t ctas = kv + (qw + AK_WARPS - 1) / AK_WARPS;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    p.kv_ctas = static_cast<unsigned>(kv);
    const cudaError_t e = d_h == 64   ? launch<64, 2>(p, ctas, stream)
                          : p.x.cu ? launch<128, 3>(p, ctas, stream)
                                   : launch<128, 2>(p, ctas, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qkq
