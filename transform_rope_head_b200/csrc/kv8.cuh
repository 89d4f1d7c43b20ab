// The paged 8-bit key/value cache (KV8): what its kernels share.
//
// Codes are e4m3, [page][key head][token of the page][channel], one fp32 step per page and key
// head (a power of two where append_kv8 wrote it).  A sequence's pages are listed in its row of
// the block table; its cached length counts this call's new tokens, which are its last ones.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace qkq {

constexpr int ST_CACHE_INDEX = 128;

// A sequence of the batch as the index tensors give it.
struct KV8Seq {
    int q0;   // its first new token's row
    int n;    // its new tokens
    int len;  // its cached tokens, the new ones included
    bool ok;  // row range and length inside the buffers
};

// cu == nullptr: one new token per sequence.
__device__ __forceinline__ KV8Seq kv8_seq(const KV8Index &x, int b)
{
    KV8Seq s;
    s.q0 = x.cu ? __ldg(x.cu + b) : b;
    s.n = x.cu ? __ldg(x.cu + b + 1) - s.q0 : 1;
    s.len = __ldg(x.seq_lens + b);
    s.ok = s.q0 >= 0 && s.n >= 0 && static_cast<int64_t>(s.q0) + s.n <= x.T && s.len >= 0 &&
           s.len <= static_cast<int64_t>(x.max_pages) << x.page_shift;
    return s;
}

// The page id of page `pi` of sequence b, -1 if it is outside the cache.  pi < max_pages.
__device__ __forceinline__ int kv8_page(const KV8Index &x, int b, int pi)
{
    const int id = __ldg(x.block_table + static_cast<int64_t>(b) * x.max_pages + pi);
    return id >= 0 && id < x.num_pages ? id : -1;
}

// Largest i in [0, count) with f(i) <= v, for f nondecreasing and f(0) <= v (else 0), by the
// whole warp: each round splits the range in 32.
template <typename F>
__device__ __forceinline__ int warp_upper(int count, int64_t v, int lane, F f)
{
    int lo = 0, n = count;
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const int i = lo + lane * step;
        const bool in = lane * step < n && f(i) <= v;
        const unsigned m = __ballot_sync(FULL_MASK, in) | 1u;
        const int k = 31 - __clz(m);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// Two 16-bit floats of one word as fp32 (bf16, or fp16 when half).
__device__ __forceinline__ float2 unpack16(uint32_t w, bool half)
{
    if (half) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool half)
{
    if (half) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Two e4m3 codes (low byte first) as an fp16 pair: exact, every e4m3 value is an fp16 value.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t pair16)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(pair16)));
    return r;
}

// Four bytes' high bits set where the byte is an e4m3 NaN code (0x7f or 0xff).
__device__ __forceinline__ uint32_t e4m3_nan_bits(uint32_t w)
{
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float lg2(float x)
{
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Steps outside [2^-40, 2^40] (and NaN) are read as the nearest end.
constexpr float KV8_STEP_MIN = 9.094947017729282e-13f, KV8_STEP_MAX = 1099511627776.0f;
__device__ __forceinline__ float kv8_step(const float *s, int64_t i)
{
    return fminf(fmaxf(__ldg(s + i), KV8_STEP_MIN), KV8_STEP_MAX);
}

}  // namespace qkq
