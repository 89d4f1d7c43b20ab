// Attention over the paged 8-bit cache on the 5th-generation tensor cores, for prompts and pieces of
// prompts (the mathematics and the work split: attention_kv8.cu).
//
// A unit is 256 query rows (tokens x heads of one key head) of a sequence, two M = 128 tiles that
// share every tile of 128 cached tokens.  Per tile of tokens and query tile
//   S [128 x 128] = Q K^T            tcgen05.mma kind::f16, both operands in shared memory
//   P = 2^(S c_j + log2 vs_j - m)    one thread per row, S read from tensor memory
//   O [128 x d_h] += P V             tcgen05.mma with P in tensor memory, over S's upper columns
// with fp32 accumulators.  The codes become fp16 on their way to shared memory (exact), rows of
// tokens for K and V alike in the 128-byte swizzle (V is read channels-major).
//
// Warps: 0-3 and 4-7 one query tile each (a thread a row: no exchange for maxima or sums), 8-11
// load and convert K and V two tiles ahead, 13-15 scale the next unit's queries into fp16, one
// thread of warp 12 issues the MMAs in the order
//   S0(i) S1(i) | PV0(i) S0(i+1) PV1(i) S1(i+1) | ...
// so that the tensor cores work on one tile while the other's exponentials are taken.
//
// A row's thread reads S twice, for the maximum and for the exponentials, in chunks of 32 columns
// and rolled loops: the roles together have to fit the instruction caches (fully unrolled, their
// warps spent more time waiting for instructions than in any pipe).
//
// The maximum is an integer and moves only when a logit passes it by more than 2^8, so rescaling
// what was summed is rare, exact, and can be done to what is already stored.
#include <limits.h>

#include "attention_kv8.cuh"
#include "tcgen05.cuh"

namespace qkq {

namespace {

constexpr int TS = 128;            // cached tokens of a tile
constexpr int TC_THREADS = 16 * 32;
constexpr int CONV0 = 8 * 32;      // first converting thread
constexpr int QLOAD0 = 13 * 32, QLOAD_WARPS = 3;
constexpr int RING = 4;            // tiles whose steps are kept
constexpr int BLOCK = 128 * 128;   // bytes of 64 channels of 128 rows
template <int DH>
constexpr int QBUF = DH == 64 ? 2 : 1;  // units whose queries are held: what shared memory has room for

template <int DH>
struct __align__(1024) TcSmem {
    uint8_t k[2][DH / 64][BLOCK];
    uint8_t v[2][DH / 64][BLOCK];
    uint8_t q[QBUF<DH>][2][DH / 64][BLOCK];
    float4 step[RING][8];                           // per 16 tokens: key step, log2 and inverse of the value step
    int2 tile[RING];                                // first token; whether every row sees all of the tile
    float fac[2][256];                              // per unit and row: what a product is times to be a base-2 logit
    int nan_unit[4];                                // number + 1 of the unit whose masked tiles hold NaN values
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t q_full[QBUF<DH>][2], q_empty[QBUF<DH>][2], s_full[2], p_full[2], o_done[2], drain;
    uint32_t tmem;
    KV8Start start;
};

__device__ __forceinline__ constexpr uint32_t idesc_f16(int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// D (tmem) (+)= A (tmem, fp16 pairs) * B (smem desc)^T
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

#define QKQ_R16(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7]), \
    "r"(r[o + 8]), "r"(r[o + 9]), "r"(r[o + 10]), "r"(r[o + 11]), "r"(r[o + 12]), "r"(r[o + 13]), "r"(r[o + 14]), "r"(r[o + 15])
#define QKQ_W16(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7]), \
    "=r"(r[o + 8]), "=r"(r[o + 9]), "=r"(r[o + 10]), "=r"(r[o + 11]), "=r"(r[o + 12]), "=r"(r[o + 13]), "=r"(r[o + 14]), "=r"(r[o + 15])

// 32 columns of this thread's lane, not waited for.
__device__ __forceinline__ void tmem_ld32_async(uint32_t a, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : QKQ_W16(r, 0), QKQ_W16(r, 16)
                 : "r"(a)
                 : "memory");
}
// The loads above have landed; the registers are tied in so that nothing reads them before.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(a),
                 QKQ_R16(r, 0)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : QKQ_W16(r, 0)
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A bounded wait by whole warps: the lanes go on, or give up, together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity)
{
    return __any_sync(FULL_MASK, mbar_wait_bounded(bar, parity));
}

// Registers per thread of the warpgroups, 128 at launch: 2 x 136 + 128 + 112 = 4 x 128.
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Every row of a unit sees every token of the tile at tok0.
__device__ __forceinline__ bool all_visible(const AttnKV8Params &p, const KV8Span &span, int tok0)
{
    return tok0 + TS - 1 <= span.first && (p.window == 0 || tok0 > span.last - p.window || tok0 + TS - 1 < p.sinks);
}

// The units of a CTA's part, each warp role on its own.
struct Units {
    int64_t cur, hi;
    int b, qt, hk, j0, j1, number;
    KV8Seq s;
    KV8Span span;
    int rows;

    __device__ __forceinline__ Units(const KV8Start &st) : cur(st.lo), hi(st.hi), b(st.b), qt(st.qt), hk(st.hk), j0(st.j0), number(0) {}
    __device__ __forceinline__ bool open(const AttnKV8Params &p)
    {
        if (cur >= hi) return false;
        s = kv8_seq_checked(p.x, b);
        span = unit_span<TS>(p, s, qt, KV8_TC_ROWS);
        j1 = static_cast<int>(min(static_cast<int64_t>(span.count), j0 + (hi - cur)));
        rows = min(KV8_TC_ROWS, s.n * p.ratio - qt * KV8_TC_ROWS);
        return true;
    }
    __device__ __forceinline__ void close(const AttnKV8Params &p)
    {
        cur += j1 - j0;
        j0 = 0;
        ++number;
        if (j1 == span.count && cur < hi) next_unit(p, s, KV8_TC_ROWS, b, qt, hk);
    }
    __device__ __forceinline__ int token(int j) const { return TS * (j < span.head ? j : j + span.skip); }
    __device__ __forceinline__ bool full(const AttnKV8Params &p, int tok0) const { return all_visible(p, span, tok0); }
};

// Channels 8 c8 .. of a Q, K or V row: 64-channel block and 16-byte place in it.  With 128 channels the block
// is which half of 16 channels it is, so that the 8 lanes that convert a row's 16-byte loads
// store to 8 different places of one 128-byte line.
template <int DH>
__device__ __forceinline__ uint32_t row_offset(int r, int c8)
{
    const int blk = DH == 128 ? (c8 & 1) : 0, place = DH == 128 ? (c8 >> 1) : c8;
    return static_cast<uint32_t>(blk * BLOCK + r * 128 + ((place ^ (r & 7)) << 4));
}

// The channel that stands at column n (a multiple of 8) of O.
template <int DH>
__device__ __forceinline__ int column_channel(int n)
{
    return DH == 128 ? 16 * ((n >> 3) & 7) + 8 * (n >> 6) : n;
}

template <int DH>
__device__ __forceinline__ bool convert_role(const AttnKV8Params &p, TcSmem<DH> &sm, int &flags)
{
    constexpr int LPR = DH / 16;       // lanes per row
    constexpr int IT = LPR;            // rows per thread, 128 / LPR apart
    const int tid = threadIdx.x - CONV0, lane = tid & 31;
    const int kc = tid % LPR, kr = tid / LPR;
    const int in_slice = (kr & 15) * DH + 16 * kc;  // the thread's bytes within any 16-token slice
    const uint32_t dst0 = row_offset<DH>(kr, 2 * kc), dst1 = row_offset<DH>(kr, 2 * kc + 1);
    int n = 0;  // tiles so far
    Units u(sm.start);
    uint4 kw[IT], vw[IT];
    float ks = 0.0f, vs = 0.0f;
    int id = -1;            // in lanes 0-7: the page of each slice of the tile being loaded, as the table has it
    int64_t at = 0;         // in lanes 0-7: where the slice begins in the cache's codes
    uint32_t none = 0;      // slices without a page (nothing cached there, or a bad page)

    auto page_id = [&](int j) {
        const int tok = u.token(j) + 16 * (lane & 7);
        return j < u.j1 && tok < u.s.len ? __ldg(p.x.block_table + static_cast<int64_t>(u.b) * p.x.max_pages + (tok >> p.x.page_shift)) : -1;
    };
    // tile j's slices, from the page ids (loaded before)
    auto locate = [&](int j) {
        const int tok = u.token(j) + 16 * (lane & 7);
        const bool ok = id >= 0 && id < p.x.num_pages;
        if (!ok && tok < u.s.len) flags |= ST_CACHE_INDEX;
        none = __ballot_sync(FULL_MASK, !ok) & 0xffu;
        const int64_t ph = static_cast<int64_t>(ok ? id : 0) * p.Hkv + u.hk;
        at = ((ph << p.x.page_shift) + (tok & ((1 << p.x.page_shift) - 1))) * DH;
        if (tid < 8) {
            ks = __ldg(p.k_steps + ph);
            vs = __ldg(p.v_steps + ph);
        }
    };
    auto load = [&](uint4 (&w)[IT], const uint8_t *codes) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int64_t slice = __shfl_sync(FULL_MASK, at, (kr >> 4) + i * (8 / IT));
            w[i] = __ldg(reinterpret_cast<const uint4 *>(codes + slice + in_slice));
        }
    };
    // rows of slices that `gone` names, and rows from `end` on, become zero
    auto clear = [&](uint4 (&w)[IT], uint32_t gone, int end) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = kr + i * (128 / LPR);
            if (((gone >> (r >> 4)) & 1) || r >= end) w[i] = make_uint4(0, 0, 0, 0);
        }
    };
    auto store = [&](uint8_t *dst, const uint4 (&w)[IT]) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[2 * k] = e4m3x2_to_half2(x[k] & 0xffffu);
                h[2 * k + 1] = e4m3x2_to_half2(x[k] >> 16);
            }
            *reinterpret_cast<uint4 *>(dst + dst0 + i * (128 / LPR) * 128) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(dst + dst1 + i * (128 / LPR) * 128) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
    };

    bool more = u.open(p);
    int j = u.j0;
    if (more) {
        id = page_id(j);
        locate(j);
        load(kw, p.k_codes);
        load(vw, p.v_codes);
        id = page_id(j + 1);
    }
    while (more) {
        const int st = n & 1;
        const uint32_t par = ((n >> 1) & 1) ^ 1;
        const int tok0 = u.token(j), end = u.s.len - tok0, number = u.number;
        const bool full = u.full(p, tok0);
        const uint32_t gone = none;
        if (!warp_wait(smem_addr(&sm.k_empty[st]), par)) return false;
        if (tid < 8) {
            const bool here = !((none >> tid) & 1);
            const float k1 = fminf(fmaxf(ks, KV8_STEP_MIN), KV8_STEP_MAX), v1 = fminf(fmaxf(vs, KV8_STEP_MIN), KV8_STEP_MAX);
            sm.step[n % RING][tid] = make_float4(here ? k1 : 0.0f, here ? lg2(v1) : -INFINITY, here ? 1.0f / v1 : 0.0f, 0.0f);
            if (tid == 0) sm.tile[n % RING] = make_int2(tok0, full);
        }
        if (gone) clear(kw, gone, 128);
        store(&sm.k[st][0][0], kw);
        if (lane == 0) mbar_arrive(smem_addr(&sm.k_full[st]));
        // on to the next tile, of this unit or the next one
        if (++j == u.j1) {
            u.close(p);
            more = u.open(p);
            j = u.j0;
            if (more) id = page_id(j);
        }
        if (more) {
            locate(j);
            load(kw, p.k_codes);
            id = page_id(j + 1);
        }
        if (!full) {
            clear(vw, gone, end);
            // NaN value codes that some row must not see (0 * NaN): out of the sums; the rows that
            // see them are looked after at the unit's end
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                uint32_t x[4] = {vw[i].x, vw[i].y, vw[i].z, vw[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t nb = e4m3_nan_bits(x[k]) >> 7;
                    x[k] &= ~(nb * 0xffu);
                    any |= nb;
                }
                vw[i] = make_uint4(x[0], x[1], x[2], x[3]);
            }
            if (any) *reinterpret_cast<volatile int *>(&sm.nan_unit[number & 3]) = number + 1;
        } else if (gone) {
            clear(vw, gone, 128);
        }
        if (!warp_wait(smem_addr(&sm.v_empty[st]), par)) return false;
        store(&sm.v[st][0][0], vw);
        if (lane == 0) mbar_arrive(smem_addr(&sm.v_full[st]));
        if (more) load(vw, p.v_codes);
        ++n;
    }
    return true;
}

__device__ __forceinline__ uint32_t bf16_pair_to_half(uint32_t w, float f)
{
    return pack16(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f, true);
}

// Queries of the units, a row on DH / 8 lanes: fp16 as they are, bf16 scaled by a power of two per row
// into fp16's range; with the sign of the softmax scale, so that a row's factor is not negative.
template <int DH>
__device__ __forceinline__ bool query_role(const AttnKV8Params &p, TcSmem<DH> &sm)
{
    constexpr int LPR = DH / 8, RPW = 32 / LPR, STRIDE = QLOAD_WARPS * RPW, BATCH = 6;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x - QLOAD0) >> 5;
    const int c8 = lane % LPR, first = warp * RPW + lane / LPR;
    const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u;
    const float scale = fabsf(p.scale_log2);
    int un[QBUF<DH>][2] = {};
    Units u(sm.start);
    for (; u.open(p); u.close(p)) {
        const int buf = u.number % QBUF<DH>;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (t * 128 >= u.rows) break;
            const int rows = min(128, u.rows - t * 128);
            int &turn = un[QBUF<DH> == 1 ? 0 : buf][t];
            const int rr0 = u.qt * KV8_TC_ROWS + t * 128, token0 = p.div_ratio(rr0);
            const uint16_t *src = p.q + (static_cast<int64_t>(u.s.q0 + token0) * p.Hq + u.hk * p.ratio + rr0 - token0 * p.ratio) * DH + 8 * c8;
            uint8_t *dst = &sm.q[buf][t][0][0];
            bool waited = turn == 0;
#pragma unroll 1
            for (int r0 = first; r0 < 128; r0 += STRIDE * BATCH) {
                uint4 w[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int r = r0 + i * STRIDE;
                    // at most 128 tokens of 2^16 heads on: 32 bits
                    const uint32_t off = static_cast<uint32_t>(r + (p.div_ratio(rr0 + r) - token0) * (p.Hq - p.ratio)) * DH;
                    w[i] = make_uint4(0, 0, 0, 0);
                    if (r < rows) w[i] = __ldg(reinterpret_cast<const uint4 *>(src + off));
                }
                if (!waited && !warp_wait(smem_addr(&sm.q_empty[buf][t]), (turn - 1) & 1)) return false;
                waited = true;
                float up[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) up[i] = scale;
                if (!p.half) {
                    uint32_t top[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        // non-negative bf16 pairs compare as they are in the upper half, the lower one shifted there
                        const uint32_t a = w[i].x & 0x7fff7fffu, b = w[i].y & 0x7fff7fffu, c = w[i].z & 0x7fff7fffu, d = w[i].w & 0x7fff7fffu;
                        top[i] = max(max(max(a, b), max(c, d)), max(max(a << 16, b << 16), max(c << 16, d << 16)));
                    }
#pragma unroll
                    for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
                        for (int i = 0; i < BATCH; ++i) top[i] = max(top[i], __shfl_xor_sync(FULL_MASK, top[i], o));
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        // a row that is not finite stays so under any factor
                        const int e = row_exponent(__uint_as_float(min(top[i] & 0xffff0000u, 0x7f7f0000u)));
                        const float f = exp2i(-e);
                        up[i] = scale * exp2i(e);
                        w[i].x = bf16_pair_to_half(w[i].x, f);
                        w[i].y = bf16_pair_to_half(w[i].y, f);
                        w[i].z = bf16_pair_to_half(w[i].z, f);
                        w[i].w = bf16_pair_to_half(w[i].w, f);
                    }
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int r = r0 + i * STRIDE;
                    if (r < 128) {
                        *reinterpret_cast<uint4 *>(dst + row_offset<DH>(r, c8)) =
                            make_uint4(w[i].x ^ flip, w[i].y ^ flip, w[i].z ^ flip, w[i].w ^ flip);
                        if (c8 == 0) sm.fac[u.number & 1][t * 128 + r] = up[i];
                    }
                }
            }
            ++turn;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.q_full[buf][t]));
        }
    }
    return true;
}

template <int DH>
__device__ __forceinline__ bool mma_role(const AttnKV8Params &p, TcSmem<DH> &sm, uint32_t tmem)
{
    const uint32_t id_s = idesc_f16(TS), id_o = idesc_f16(DH) | (1u << 16);  // V: channels-major
    // K, Q: rows of 64 channels, 8-row groups 1024 bytes apart; V: 64 channels of a token a row, 8-token
    // groups 1024 bytes, 64-channel blocks BLOCK bytes apart
    const uint64_t q0 = sw128_desc(smem_addr(&sm.q[0][0][0][0])), k0 = sw128_desc(smem_addr(&sm.k[0][0][0]));
    const uint64_t v0 = (sw128_desc(smem_addr(&sm.v[0][0][0])) & ~(0x3fffull << 16)) | (static_cast<uint64_t>(BLOCK >> 4) << 16);
    constexpr uint64_t STAGE = (DH / 64) * (BLOCK >> 4);
    int n = 0, cnt[2] = {0, 0}, un[QBUF<DH>][2] = {};  // tiles; tiles and units of each query tile
    Units u(sm.start);
    while (u.open(p)) {
        const int last_t = u.rows > 128 ? 1 : 0, buf = u.number % QBUF<DH>;
#pragma unroll 1
        for (int j = u.j0; j <= u.j1; ++j, ++n) {
            // tile j - 1's values, then tile j's scores (which take the columns that P leaves)
            const int st = n & 1;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (t > last_t) break;
                if (j > u.j0) {
                    if (t == 0 && !mbar_wait_bounded(smem_addr(&sm.v_full[st ^ 1]), ((n - 1) >> 1) & 1)) return false;
                    if (!mbar_wait_bounded(smem_addr(&sm.p_full[t]), cnt[t] & 1)) return false;
                    ++cnt[t];
                    tc_fence_after();
                    const uint64_t v = v0 + (st ^ 1) * STAGE;
#pragma unroll
                    for (int s = 0; s < TS / 16; ++s)
                        mma_f16_ts(tmem + 2 * TS + t * DH, tmem + t * TS + TS / 2 + 8 * s, v + s * (16 * 128 >> 4), id_o,
                                   s || j - 1 > u.j0 ? 1u : 0u);
                    if (t == last_t) mma_commit(smem_addr(&sm.v_empty[st ^ 1]));
                    if (j == u.j1) mma_commit(smem_addr(&sm.o_done[t]));
                } else {
                    int &turn = un[QBUF<DH> == 1 ? 0 : buf][t];
                    if (!mbar_wait_bounded(smem_addr(&sm.q_full[buf][t]), turn & 1)) return false;
                    ++turn;
                }
                if (j < u.j1) {
                    if (t == 0 && !mbar_wait_bounded(smem_addr(&sm.k_full[st]), (n >> 1) & 1)) return false;
                    tc_fence_after();
                    const uint64_t q = q0 + (2 * buf + t) * STAGE, k = k0 + st * STAGE;
#pragma unroll
                    for (int s = 0; s < DH / 16; ++s) {
                        const uint32_t off = ((s >> 2) * BLOCK + (s & 3) * 32) >> 4;
                        mma_bf16(tmem + t * TS, q + off, k + off, id_s, s ? 1u : 0u);
                    }
                    // done when all before it is, the last tile's values among that
                    mma_commit(smem_addr(&sm.s_full[t]));
                    if (t == last_t) mma_commit(smem_addr(&sm.k_empty[st]));
                    if (j + 1 == u.j1) mma_commit(smem_addr(&sm.q_empty[buf][t]));
                }
            }
        }
        --n;
        u.close(p);
    }
    return true;
}

__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Which columns of a tile the row sees: those below hi, and not in [lo, ...) unless below sk.
struct RowMask {
    int hi, lo, sk;
    static __device__ __forceinline__ uint32_t below(int n)
    {
        return n >= 32 ? FULL_MASK : (1u << max(n, 0)) - 1u;
    }
    // bits of columns c0 .. c0 + 31
    __device__ __forceinline__ uint32_t bits(int c0) const { return below(hi - c0) & (~below(lo - c0) | below(sk - c0)); }
};

// The largest base-2 logit (without the maximum's offset) of 32 columns.
template <bool MASKED>
__device__ __forceinline__ float chunk_top(const uint32_t (&raw)[32], const float4 *step, float fac, uint32_t bits)
{
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = __uint_as_float(raw[16 * g + i]);
            if (MASKED && !((bits >> (16 * g + i)) & 1)) x[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 1; i < 16; ++i) x[0] = fmaxf(x[0], x[i]);
        // the factor is not negative and rounding keeps order: the logit of the maximum
        top = fmaxf(top, __fmaf_rn(x[0], fac * step[g].x, step[g].y));
    }
    return top;
}

// P of 32 columns as fp16 pairs, and their part of the row's sum.
template <bool MASKED>
__device__ __forceinline__ void chunk_p(const uint32_t (&raw)[32], const float4 *step, float fac, float m, uint32_t bits,
                                        uint32_t (&pw)[16], float &l)
{
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const float f = fac * step[g].x, a = step[g].y - m;
        const uint64_t f2 = pair(f, f), a2 = pair(a, a);
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = 16 * g + 2 * i;
            float x, y;
            unpair(fma_pair(pair(__uint_as_float(raw[k]), __uint_as_float(raw[k + 1])), f2, a2), x, y);
            x = ex2(x);
            y = ex2(y);
            if (MASKED) {
                x = (bits >> k) & 1 ? x : 0.0f;
                y = (bits >> (k + 1)) & 1 ? y : 0.0f;
            }
            sum = add_pair(sum, pair(x, y));
            pw[8 * g + i] = pack16(x, y, true);
        }
        float x, y;
        unpair(sum, x, y);
        l = __fmaf_rn(x + y, step[g].z, l);
    }
}

// A row's statistics: m the (whole-numbered) maximum's offset, l the sum, pass what a logit must
// exceed to move m (-inf: none seen yet).
struct RowState {
    float m, l, pass;
};

// S of one tile to P, the row's thread.
template <int DH, bool MASKED>
__device__ __forceinline__ void softmax_tile(const float4 *step, uint32_t p_full, bool first, uint32_t s_cols, uint32_t o_cols,
                                             float fac, const RowMask &mask, RowState &r)
{
    uint32_t a[32], b[32], pw[16];
    tmem_ld32_async(s_cols, a);
    tmem_ld32_async(s_cols + 32, b);
    float top = -INFINITY;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        tmem_ld_wait(a);
        tmem_ld_wait(b);
        top = fmaxf(top, chunk_top<MASKED>(a, step + 4 * h, fac, MASKED ? mask.bits(64 * h) : 0u));
        if (h == 0) tmem_ld32_async(s_cols + 64, a);
        top = fmaxf(top, chunk_top<MASKED>(b, step + 4 * h + 2, fac, MASKED ? mask.bits(64 * h + 32) : 0u));
        if (h == 0) tmem_ld32_async(s_cols + 96, b);
    }
    const bool moves = top > r.pass;
    if (__any_sync(FULL_MASK, moves)) {
        // the maximum moves: a whole number, so that every factor is a power of two (before a row's
        // first logit there is nothing to rescale)
        const float to = moves ? ceilf(top) : r.m;
        const float alpha = moves && r.pass > -INFINITY ? ex2(r.m - to) : 1.0f;
        if (moves) {
            r.m = to;
            r.pass = to + 8.0f;
        }
        r.l *= alpha;
        if (!first) {
            // the product before this tile's S has been added to O
#pragma unroll 1
            for (int k = 0; k < DH / 16; ++k) {
                uint32_t w[16];
                tmem_ld16(o_cols + 16 * k, w);
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
                tmem_st16(o_cols + 16 * k, w);
            }
        }
    }
    // backwards: the last two chunks are at hand, and P takes the upper columns once they are read
#pragma unroll 1
    for (int h = 1; h >= 0; --h) {
        if (h == 0) {
            tmem_ld_wait(a);
            tmem_ld_wait(b);
        }
        chunk_p<MASKED>(b, step + 4 * h + 2, fac, r.m, MASKED ? mask.bits(64 * h + 32) : 0u, pw, r.l);
        if (h == 1) tmem_ld32_async(s_cols + 32, b);
        tmem_st16(s_cols + TS / 2 + 32 * h + 16, pw);
        chunk_p<MASKED>(a, step + 4 * h, fac, r.m, MASKED ? mask.bits(64 * h) : 0u, pw, r.l);
        if (h == 1) tmem_ld32_async(s_cols, a);
        tmem_st16(s_cols + TS / 2 + 32 * h, pw);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(p_full);
}

// Which of the 8 channels from ch on have a NaN value code that a row at index `at` sees in tiles
// [j0, j1) of a unit that not every row sees wholly (the converting warps took those codes out).
template <int DH>
__device__ __noinline__ uint32_t nan_channels(const AttnKV8Params &p, int b, int hk, int j0, int j1, KV8Span span, int at, int ch)
{
    uint32_t m = 0;
    for (int j = j0; j < j1; ++j) {
        const int tok0 = TS * (j < span.head ? j : j + span.skip);
        if (all_visible(p, span, tok0)) continue;
        for (int tok = tok0; tok < tok0 + TS && tok <= at; ++tok) {
            if (p.window && tok <= at - p.window && tok >= p.sinks) continue;
            const int id = kv8_page(p.x, b, tok >> p.x.page_shift);
            if (id < 0) continue;
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(
                p.v_codes + (((static_cast<int64_t>(id) * p.Hkv + hk) << p.x.page_shift) + (tok & ((1 << p.x.page_shift) - 1))) * DH + ch));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m |= ((w.x >> (8 * i)) & 0x7f) == 0x7f ? 1u << i : 0u;
                m |= ((w.y >> (8 * i)) & 0x7f) == 0x7f ? 16u << i : 0u;
            }
        }
    }
    return m;
}

template <int DH>
__device__ __forceinline__ bool softmax_role(const AttnKV8Params &p, TcSmem<DH> &sm, uint32_t tmem, const KV8Partials &part)
{
    const int t = threadIdx.x >> 7, r = threadIdx.x & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(r & 96) << 16);
    const uint32_t s_cols = lanes + t * TS, o_cols = lanes + 2 * TS + t * DH;
    int n = 0, cnt = 0, unit = 0;  // tiles of the part; tiles and units of this query tile
    Units u(sm.start);
    for (; u.open(p); u.close(p)) {
        if (t * 128 >= u.rows) {
            n += u.j1 - u.j0;
            continue;
        }
        const int row = t * 128 + r;
        const bool live = row < u.rows;
        const int rr = u.qt * KV8_TC_ROWS + row;
        const int token = p.div_ratio(rr), at = live ? u.s.len - u.s.n + token : -1;
        RowState st{0.0f, 0.0f, -INFINITY};
        float fac = 0.0f;
#pragma unroll 1
        for (int j = u.j0; j < u.j1; ++j, ++n, ++cnt) {
            if (!warp_wait(smem_addr(&sm.s_full[t]), cnt & 1)) return false;
            tc_fence_after();
            const bool first = j == u.j0;
            if (first) fac = sm.fac[u.number & 1][row];
            const int2 tile = sm.tile[n % RING];
            const int hi = at - tile.x + 1;
            const RowMask mask{hi, p.window ? hi - p.window : 0, p.window ? p.sinks - tile.x : 0};
            const uint32_t p_full = smem_addr(&sm.p_full[t]);
            if (tile.y)
                softmax_tile<DH, false>(sm.step[n % RING], p_full, first, s_cols, o_cols, fac, mask, st);
            else
                softmax_tile<DH, true>(sm.step[n % RING], p_full, first, s_cols, o_cols, fac, mask, st);
        }

        // ---- the unit's end ------------------------------------------------------------------------
        if (!warp_wait(smem_addr(&sm.o_done[t]), unit & 1)) return false;
        ++unit;
        tc_fence_after();
        const bool whole = u.j0 == 0 && u.j1 == u.span.count;
        const bool nan = *reinterpret_cast<volatile int *>(&sm.nan_unit[u.number & 3]) == u.number + 1;
        const bool empty = st.pass == -INFINITY && st.l == 0.0f;
        const float top = st.pass == -INFINITY ? -INFINITY : st.m;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (u.number == 0 ? 0 : 1);
        const int64_t q_row = static_cast<int64_t>(u.s.q0) * p.Hq + u.hk * p.ratio + rr + static_cast<int64_t>(token) * (p.Hq - p.ratio);
        const float inv = empty ? 0.0f : 1.0f / st.l;
#pragma unroll 1
        for (int c = 0; c < DH; c += 32) {
            uint32_t raw[32];
            tmem_ld32_async(o_cols + c, raw);
            tmem_ld_wait(raw);
            if (!live) continue;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int ch = column_channel<DH>(c + 8 * g);
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(raw[8 * g + i]);
                if (nan) {
                    const uint32_t bad = nan_channels<DH>(p, u.b, u.hk, u.j0, u.j1, u.span, at, ch);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = (bad >> i) & 1 ? __uint_as_float(0x7fc00000u) : o[i];
                }
                if (whole) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = empty ? 0u : pack16(o[2 * i] * inv, o[2 * i + 1] * inv, p.half);
                    *reinterpret_cast<uint4 *>(p.out + q_row * DH + ch) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(part.o + (slot * KV8_TC_ROWS + row) * DH + ch);
                    dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                    dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                }
            }
        }
        if (live && whole && p.lse) p.lse[q_row] = empty ? -INFINITY : (lg2(st.l) + top) * 0.6931471805599453f;
        if (live && !whole) *reinterpret_cast<float2 *>(part.ml + (slot * KV8_TC_ROWS + row) * 2) = make_float2(top, st.l);
        tc_fence_before();
    }
    return true;
}

template <int DH>
__global__ void __launch_bounds__(TC_THREADS, 1) k_attention_kv8_tc(const __grid_constant__ AttnKV8Params p)
{
    extern __shared__ uint8_t smem_raw[];
    TcSmem<DH> &sm = *reinterpret_cast<TcSmem<DH> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_prior_grid();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sm.k_full[i]), 4);
            mbar_init(smem_addr(&sm.v_full[i]), 4);
            mbar_init(smem_addr(&sm.k_empty[i]), 1);
            mbar_init(smem_addr(&sm.v_empty[i]), 1);
#pragma unroll
            for (int b = 0; b < QBUF<DH>; ++b) {
                mbar_init(smem_addr(&sm.q_full[b][i]), QLOAD_WARPS);
                mbar_init(smem_addr(&sm.q_empty[b][i]), 1);
            }
            mbar_init(smem_addr(&sm.s_full[i]), 1);
            mbar_init(smem_addr(&sm.p_full[i]), 4);
            mbar_init(smem_addr(&sm.o_done[i]), 1);
        }
        mbar_init(smem_addr(&sm.drain), 1);
        fence_mbar_init();
#pragma unroll
        for (int i = 0; i < 4; ++i) sm.nan_unit[i] = 0;
    }
    if (warp == 12) {
        tmem_alloc(smem_addr(&sm.tmem), 512);
        tmem_relinquish();
    }
    find_start<TS, KV8_TC_ROWS, TC_THREADS>(p, sm.start, 1);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    allow_next_grid();  // after the allocation: a later grid's must not come first
    const uint32_t tmem = sm.tmem;
    const KV8Partials part(p.workspace, gridDim.x, KV8_TC_ROWS, DH);
    if (threadIdx.x == 0)
        part.meta[blockIdx.x] = KV8Meta{sm.start.lo, sm.start.hi > sm.start.lo ? sm.start.j0 : 0, sm.start.b, sm.start.qt, sm.start.hk};

    int flags = threadIdx.x == 0 ? sm.start.flags : 0;
    bool ok = true;
    if (warp < 8) {
        more_registers<136>();
        ok = softmax_role<DH>(p, sm, tmem, part);
    } else if (warp < 12) {
        fewer_registers<128>();
        ok = convert_role<DH>(p, sm, flags);
    } else {
        fewer_registers<112>();
        if (warp > 12) {
            ok = query_role<DH>(p, sm);
        } else if (lane == 0) {
            ok = mma_role<DH>(p, sm, tmem);
            // nothing of this CTA runs on when its tensor memory goes
            mma_commit(smem_addr(&sm.drain));
            ok &= mbar_wait_bounded(smem_addr(&sm.drain), 0);
        }
        __syncwarp();
    }
    if (!ok) flags |= ST_TIMEOUT;
    if (p.status && flags) atomicOr(p.status, flags);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DH>
cudaError_t launch(const AttnKV8Params &p, const DeviceInfo &dev, cudaStream_t stream)
{
    constexpr int smem = sizeof(TcSmem<DH>) + 1024;
    const cudaError_t e = cudaFuncSetAttribute(k_attention_kv8_tc<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int ctas = dev.num_sms < KV8_TC_MAX_CTAS ? dev.num_sms : KV8_TC_MAX_CTAS;
    const cudaError_t f = launch_after_prior(k_attention_kv8_tc<DH>, dim3(ctas), dim3(TC_THREADS), smem, stream, p);
    if (f != cudaSuccess) return f;
    return attention_kv8_join_launch(p, DH, ctas, KV8_TC_ROWS, stream);
}

}  // namespace

cudaError_t attention_kv8_tc_launch(const AttnKV8Params &p, int d_h, const DeviceInfo &dev, cudaStream_t stream)
{
    const cudaError_t e = d_h == 64 ? launch<64>(p, dev, stream) : launch<128>(p, dev, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qkq
