// Attention over the paged 8-bit cache on the 5th-generation tensor cores, for prompts and pieces of
// prompts (the mathematics and the work split: attention_kv8.cu).
//
// A unit is 256 query rows (tokens x heads of one key head) of a sequence, two M = 128 tiles that
// share every tile of 128 cached tokens.  Per tile of tokens and query tile
//   S [128 x 128] = Q K^T            tcgen05.mma kind::f16, both operands in shared memory
//   P = 2^(S c_j + log2 vs_j - m)    one thread per row, S read from tensor memory
//   O [128 x d_h] += P V             tcgen05.mma with P in tensor memory, over S's own columns
// with fp32 accumulators.  The codes become fp16 on their way to shared memory (exact), K as rows of
// tokens, V transposed to rows of channels, both in the 128-byte swizzle.
//
// Warps: 0-3 and 4-7 one query tile each (a thread a row: no exchange for maxima or sums), 8-11
// load and convert K and V two tiles ahead, one thread of warp 12 issues the MMAs (warps 13-15 only
// complete its warpgroup, which gives up registers) in the order
//   S0(i) S1(i) | PV0(i) S0(i+1) PV1(i) S1(i+1) | ...
// so that the tensor cores work on one tile while the other's exponentials are taken.
//
// The maximum is an integer and moves only when a logit passes it by more than 2^8, so rescaling
// what was summed is rare, exact, and can be done to what is already stored.
#include "attention_kv8.cuh"
#include "tcgen05.cuh"

namespace qkq {

namespace {

constexpr int TS = 128;            // cached tokens of a tile
constexpr int TC_THREADS = 16 * 32;
constexpr int CONV0 = 8 * 32;      // first converting thread
constexpr int RING = 4;            // tiles whose steps are kept

template <int DH>
struct __align__(1024) TcSmem {
    uint8_t q[2][DH / 64][128 * 128];
    uint8_t k[2][DH / 64][128 * 128];
    uint8_t v[2][2][DH * 128];
    float ks[RING][8], lvs[RING][8], ivs[RING][8];  // per 16 tokens
    int nan_unit[4];                                // number + 1 of the unit whose masked tiles hold NaN values
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t q_full[2], s_full[2], p_full[2], o_done[2], drain;
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

// Registers per thread of the warpgroups, 128 at launch: 2 x 152 + 128 + 80 = 4 x 128.
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

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
    // every row of the unit sees every token of the tile at tok0
    __device__ __forceinline__ bool full(const AttnKV8Params &p, int tok0) const
    {
        return tok0 + TS - 1 <= span.first && (p.window == 0 || tok0 > span.last - p.window || tok0 + TS - 1 < p.sinks);
    }
};

// Channel ch of a Q or K row: 64-channel block and 16-byte place in it.  With 128 channels the block is
// which half of 16 channels it is in, so that the 8 lanes that convert a row's 16-byte loads
// store to 8 different places of one 128-byte line.
template <int DH>
__device__ __forceinline__ uint32_t row_offset(int r, int c8)
{
    const int blk = DH == 128 ? (c8 & 1) : 0, place = DH == 128 ? (c8 >> 1) : c8;
    return static_cast<uint32_t>(blk * 128 * 128 + r * 128 + ((place ^ (r & 7)) << 4));
}

template <int DH>
__device__ __forceinline__ bool convert_role(const AttnKV8Params &p, TcSmem<DH> &sm, int &flags)
{
    constexpr int LPR = DH / 16;       // lanes per K row
    constexpr int KIT = LPR;           // K iterations: 128 / LPR rows each
    constexpr int VB = DH / 8;         // V bytes per token and lane
    constexpr int VW = VB / 4;
    const int tid = threadIdx.x - CONV0, lane = tid & 31;
    const int kc = tid % LPR, kr = tid / LPR;
    const int tgl = tid & 7, vc = (tid >> 3) & 7, tgh = tid >> 6;
    const int64_t mask = (1 << p.x.page_shift) - 1;
    int n = 0;  // tiles so far
    Units u(sm.start);
    uint4 kw[KIT];
    uint32_t vw[8][VW];

    // page of each 16-token slice of a tile, in lanes 0-7
    auto pages = [&](int j) {
        const int tok = u.token(j) + 16 * (lane & 7);
        if (j >= u.j1 || tok >= u.s.len) return -1;
        const int id = kv8_page(p.x, u.b, tok >> p.x.page_shift);
        if (id < 0) flags |= ST_CACHE_INDEX;
        return id;
    };
    auto load_k = [&](int j, int pg) {
        const int tok0 = u.token(j);
#pragma unroll
        for (int i = 0; i < KIT; ++i) {
            const int r = kr + i * (128 / LPR);
            const int id = __shfl_sync(FULL_MASK, pg, r >> 4);
            kw[i] = make_uint4(0, 0, 0, 0);
            if (id >= 0) {
                const int64_t row = ((static_cast<int64_t>(id) * p.Hkv + u.hk) << p.x.page_shift) + ((tok0 + r) & mask);
                kw[i] = __ldg(reinterpret_cast<const uint4 *>(p.k_codes + row * DH + 16 * kc));
            }
        }
    };
    auto load_v = [&](int j, int pg) {
        const int tok0 = u.token(j) + 64 * tgh + 8 * tgl;
        const int id = __shfl_sync(FULL_MASK, pg, 4 * tgh + (tgl >> 1));
        const int64_t row = ((static_cast<int64_t>(id) * p.Hkv + u.hk) << p.x.page_shift) + (tok0 & mask);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int w = 0; w < VW; ++w) vw[i][w] = 0;
            if (id >= 0 && tok0 + i < u.s.len) {
                const uint8_t *src = p.v_codes + (row + i) * DH + VB * vc;
                if (DH == 128) {
                    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src));
                    vw[i][0] = x.x;
                    vw[i][1] = x.y;
                    vw[i][VW - 2] = x.z;
                    vw[i][VW - 1] = x.w;
                } else {
                    const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src));
                    vw[i][0] = x.x;
                    vw[i][1] = x.y;
                }
            }
        }
    };

    bool more = u.open(p);
    int pg = -1;
    if (more) {
        pg = pages(u.j0);
        load_k(u.j0, pg);
        load_v(u.j0, pg);
    }
    while (more) {
        for (int j = u.j0; j < u.j1; ++j, ++n) {
            const int st = n & 1;
            const uint32_t par = ((n >> 1) & 1) ^ 1;
            const int tok0 = u.token(j);
            const bool last = j + 1 == u.j1;
            const int pg_next = last ? -1 : pages(j + 1);
            // steps of the tile's slices
            float ks = 0.0f, vs = 1.0f;
            if (tid < 8 && pg >= 0) {
                const int64_t ph = static_cast<int64_t>(pg) * p.Hkv + u.hk;
                ks = kv8_step(p.k_steps, ph);
                vs = kv8_step(p.v_steps, ph);
            }
            if (!warp_wait(smem_addr(&sm.k_empty[st]), par)) return false;
            if (tid < 8) {
                sm.ks[n % RING][tid] = ks;
                sm.lvs[n % RING][tid] = pg >= 0 ? lg2(vs) : -INFINITY;
                sm.ivs[n % RING][tid] = pg >= 0 ? 1.0f / vs : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < KIT; ++i) {
                const int r = kr + i * (128 / LPR);
                const uint32_t x[4] = {kw[i].x, kw[i].y, kw[i].z, kw[i].w};
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<uint4 *>(&sm.k[st][0][0] + row_offset<DH>(r, 2 * kc + h)) =
                        make_uint4(e4m3x2_to_half2(x[2 * h] & 0xffffu), e4m3x2_to_half2(x[2 * h] >> 16),
                                   e4m3x2_to_half2(x[2 * h + 1] & 0xffffu), e4m3x2_to_half2(x[2 * h + 1] >> 16));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.k_full[st]));
            if (!last) load_k(j + 1, pg_next);

            if (!u.full(p, tok0)) {
                // NaN value codes that some row must not see (0 * NaN): out of the sums; the rows that
                // see them are looked after at the unit's end
                uint32_t any = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        const uint32_t nb = e4m3_nan_bits(vw[i][w]) >> 7;
                        vw[i][w] &= ~(nb * 0xffu);
                        any |= nb;
                    }
                if (any) *reinterpret_cast<volatile int *>(&sm.nan_unit[u.number & 3]) = u.number + 1;
            }
            if (!warp_wait(smem_addr(&sm.v_empty[st]), par)) return false;
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a[4], b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x = __byte_perm(vw[2 * i][w], vw[2 * i + 1][w], h ? 0x7362 : 0x5140);
                        a[i] = e4m3x2_to_half2(x & 0xffffu);
                        b[i] = e4m3x2_to_half2(x >> 16);
                    }
                    const int ch = VB * vc + 4 * w + 2 * h;
                    uint8_t *dst = &sm.v[st][tgh][0] + ch * 128;
                    *reinterpret_cast<uint4 *>(dst + ((tgl ^ (ch & 7)) << 4)) = make_uint4(a[0], a[1], a[2], a[3]);
                    *reinterpret_cast<uint4 *>(dst + 128 + ((tgl ^ ((ch + 1) & 7)) << 4)) = make_uint4(b[0], b[1], b[2], b[3]);
                }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.v_full[st]));
            if (!last) load_v(j + 1, pg_next);
            pg = pg_next;
        }
        u.close(p);
        more = u.open(p);
        if (more) {
            pg = pages(u.j0);
            load_k(u.j0, pg);
            load_v(u.j0, pg);
        }
    }
    return true;
}

template <int DH>
__device__ __forceinline__ bool mma_role(const AttnKV8Params &p, TcSmem<DH> &sm, uint32_t tmem)
{
    const uint32_t id_s = idesc_f16(TS), id_o = idesc_f16(DH);
    int n = 0, cnt[2] = {0, 0}, un[2] = {0, 0};  // tiles; tiles and units of each query tile
    auto scores = [&](int t, int st, bool last_reader) {
        uint64_t q = sw128_desc(smem_addr(&sm.q[t][0][0])), k = sw128_desc(smem_addr(&sm.k[st][0][0]));
        asm volatile("" : "+l"(q), "+l"(k));  // built here, not kept in registers for every step
#pragma unroll
        for (int s = 0; s < DH / 16; ++s) {
            const uint32_t off = ((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4;
            mma_bf16(tmem + t * TS, q + off, k + off, id_s, s ? 1u : 0u);
        }
        mma_commit(smem_addr(&sm.s_full[t]));
        if (last_reader) mma_commit(smem_addr(&sm.k_empty[st]));
    };
    auto values = [&](int t, int st, bool accumulate, bool last_reader) {
        uint64_t v = sw128_desc(smem_addr(&sm.v[st][0][0]));
        asm volatile("" : "+l"(v));
#pragma unroll
        for (int s = 0; s < TS / 16; ++s)
            mma_f16_ts(tmem + 2 * TS + t * DH, tmem + t * TS + 8 * s, v + (((s >> 2) * (DH * 128) + (s & 3) * 32) >> 4), id_o,
                       accumulate || s ? 1u : 0u);
        mma_commit(smem_addr(&sm.o_done[t]));
        if (last_reader) mma_commit(smem_addr(&sm.v_empty[st]));
    };
    Units u(sm.start);
    while (u.open(p)) {
        const bool two = u.rows > 128;
        for (int t = 0; t <= (two ? 1 : 0); ++t) {
            if (!mbar_wait_bounded(smem_addr(&sm.q_full[t]), un[t] & 1)) return false;
            ++un[t];
            if (t == 0 && !mbar_wait_bounded(smem_addr(&sm.k_full[n & 1]), (n >> 1) & 1)) return false;
            tc_fence_after();
            scores(t, n & 1, t == (two ? 1 : 0));
        }
        for (int j = u.j0; j < u.j1; ++j, ++n) {
            const bool more = j + 1 < u.j1;
            const int st = n & 1, next = (n + 1) & 1;
            if (!mbar_wait_bounded(smem_addr(&sm.v_full[st]), (n >> 1) & 1)) return false;
            for (int t = 0; t <= (two ? 1 : 0); ++t) {
                const bool last = t == (two ? 1 : 0);
                if (!mbar_wait_bounded(smem_addr(&sm.p_full[t]), cnt[t] & 1)) return false;
                ++cnt[t];
                tc_fence_after();
                values(t, st, j > u.j0, last);
                if (more) {
                    if (t == 0 && !mbar_wait_bounded(smem_addr(&sm.k_full[next]), ((n + 1) >> 1) & 1)) return false;
                    tc_fence_after();
                    scores(t, next, last);
                }
            }
        }
        u.close(p);
    }
    return true;
}

template <int DH>
__device__ __forceinline__ bool softmax_role(const AttnKV8Params &p, TcSmem<DH> &sm, uint32_t tmem, const KV8Partials &part)
{
    const int t = threadIdx.x >> 7, r = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(r & 96) << 16);
    const uint32_t s_cols = lanes + t * TS, o_cols = lanes + 2 * TS + t * DH;
    int n = 0, cnt = 0;
    Units u(sm.start);
    for (; u.open(p); u.close(p)) {
        if (t * 128 >= u.rows) {
            n += u.j1 - u.j0;
            continue;
        }
        const int row = t * 128 + r;
        const bool live = row < u.rows;
        const int rr = u.qt * KV8_TC_ROWS + row;
        // ---- the row's query, scaled into fp16 -----------------------------------------------
        float fac;
        {
            uint32_t w[DH / 2];
            float amax = 0.0f;
            if (live) {
                const uint16_t *src = p.q + (static_cast<int64_t>(u.s.q0 + rr / p.ratio) * p.Hq + u.hk * p.ratio + rr % p.ratio) * DH;
#pragma unroll
                for (int i = 0; i < DH / 8; ++i) {
                    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src) + i);
                    w[4 * i] = x.x;
                    w[4 * i + 1] = x.y;
                    w[4 * i + 2] = x.z;
                    w[4 * i + 3] = x.w;
                }
#pragma unroll
                for (int i = 0; i < DH / 2; ++i) {
                    const float2 v = unpack16(w[i], p.half);
                    amax = fmaxf(amax, fabsf(v.x) <= 3.402823466e38f ? fabsf(v.x) : 0.0f);
                    amax = fmaxf(amax, fabsf(v.y) <= 3.402823466e38f ? fabsf(v.y) : 0.0f);
                }
            } else {
#pragma unroll
                for (int i = 0; i < DH / 2; ++i) w[i] = 0;
            }
            const int e = row_exponent(amax);
            const float up = exp2i(-e);
            fac = p.scale_log2 * exp2i(e);
#pragma unroll
            for (int i = 0; i < DH / 8; ++i) {
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 v = unpack16(w[4 * i + k], p.half);
                    h[k] = pack16(v.x * up, v.y * up, true);
                }
                *reinterpret_cast<uint4 *>(&sm.q[t][0][0] + row_offset<DH>(r, i)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.q_full[t]));
        }
        const int at = live ? u.s.len - u.s.n + rr / p.ratio : -1;
        float m = 0.0f, l = 0.0f, pass = -INFINITY;  // pass: what a logit must exceed to move m (-inf: none seen yet)

        for (int j = u.j0; j < u.j1; ++j, ++n, ++cnt) {
            const int tok0 = u.token(j);
            const bool full = u.full(p, tok0);
            // columns that the row sees: c <= hi and (c > lo or c < sk)
            const int hi = at - tok0, lo = p.window ? hi - p.window : -1, sk = p.sinks - tok0;
            if (!warp_wait(smem_addr(&sm.s_full[t]), cnt & 1)) return false;
            tc_fence_after();
            uint32_t buf[2][32];
            tmem_ld32_async(s_cols, buf[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t(&raw)[32] = buf[c & 1];
                tmem_ld_wait(raw);
                if (c < 3) tmem_ld32_async(s_cols + 32 * (c + 1), buf[(c + 1) & 1]);
                float x[32];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float f = fac * sm.ks[n % RING][2 * c + g], a = sm.lvs[n % RING][2 * c + g] - m;
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[16 * g + i] = __fmaf_rn(__uint_as_float(raw[16 * g + i]), f, a);
                }
                if (!full) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int col = 32 * c + i;
                        if (!(col <= hi && (col > lo || col < sk))) x[i] = -INFINITY;
                    }
                }
                float top = x[0];
#pragma unroll
                for (int i = 1; i < 32; ++i) top = fmaxf(top, x[i]);
                if (__any_sync(FULL_MASK, top > pass)) {
                    // the maximum moves: a whole number, so that every factor is a power of two
                    // (before a row's first logit there is nothing to rescale)
                    const float shift = top > pass ? ceilf(top) : 0.0f;
                    const float alpha = top > pass && pass > 0.0f ? ex2(-shift) : 1.0f;
                    if (top > pass) {
                        m += shift;
                        pass = 8.0f;
                    }
                    l *= alpha;
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] -= shift;
                    if (c > 0) {
                        const __half2 a2 = __float2half2_rn(alpha);
                        if (c < 3) tmem_ld_wait(buf[(c + 1) & 1]);
                        tmem_st_wait();
                        for (int k = 0; k < c; ++k) {
                            uint32_t w[16];
                            tmem_ld16(s_cols + 16 * k, w);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&w[i]), a2);
                                w[i] = *reinterpret_cast<const uint32_t *>(&v);
                            }
                            tmem_st16(s_cols + 16 * k, w);
                        }
                    }
                    if (j > u.j0) {
                        if (!warp_wait(smem_addr(&sm.o_done[t]), (cnt - 1) & 1)) return false;
                        tc_fence_after();
                        for (int k = 0; k < DH / 16; ++k) {
                            uint32_t w[16];
                            tmem_ld16(o_cols + 16 * k, w);
#pragma unroll
                            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
                            tmem_st16(o_cols + 16 * k, w);
                        }
                    }
                }
                uint32_t pw[16];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float a = ex2(x[16 * g + 2 * i]), b = ex2(x[16 * g + 2 * i + 1]);
                        sum += a + b;
                        pw[8 * g + i] = pack16(a, b, true);
                    }
                    l = __fmaf_rn(sum, sm.ivs[n % RING][2 * c + g], l);
                }
                tmem_st16(s_cols + 16 * c, pw);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[t]));
        }

        // ---- the unit's end ------------------------------------------------------------------------
        if (!warp_wait(smem_addr(&sm.o_done[t]), (cnt - 1) & 1)) return false;
        tc_fence_after();
        const bool whole = u.j0 == 0 && u.j1 == u.span.count;
        const bool nan = *reinterpret_cast<volatile int *>(&sm.nan_unit[u.number & 3]) == u.number + 1;
        const float top = pass == -INFINITY ? -INFINITY : m;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (u.number == 0 ? 0 : 1);
        for (int c = 0; c < DH / 32; ++c) {
            uint32_t raw[32];
            tmem_ld32_async(o_cols + 32 * c, raw);
            tmem_ld_wait(raw);
            if (nan && live) {
                for (int j = u.j0; j < u.j1; ++j) {
                    const int tok0 = u.token(j);
                    if (u.full(p, tok0)) continue;
                    for (int k = 0; k < TS && tok0 + k <= at; ++k) {
                        const int tok = tok0 + k;
                        if (p.window && tok <= at - p.window && tok >= p.sinks) continue;
                        const int id = kv8_page(p.x, u.b, tok >> p.x.page_shift);
                        if (id < 0) continue;
                        const uint8_t *src = p.v_codes + (((static_cast<int64_t>(id) * p.Hkv + u.hk) << p.x.page_shift) + (tok & ((1 << p.x.page_shift) - 1))) * DH + 32 * c;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if ((__ldg(src + i) & 0x7f) == 0x7f) raw[i] = 0x7fc00000u;
                    }
                }
            }
            if (live) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 v = make_float4(__uint_as_float(raw[4 * i]), __uint_as_float(raw[4 * i + 1]),
                                                 __uint_as_float(raw[4 * i + 2]), __uint_as_float(raw[4 * i + 3]));
                    const int ch = 32 * c + 4 * i;
                    if (whole) {
                        store_row(p, u.s, rr, u.hk, ch, DH, v, top, l);
                    } else {
                        *reinterpret_cast<float4 *>(part.o + (slot * KV8_TC_ROWS + row) * DH + ch) = v;
                        if (ch == 0) *reinterpret_cast<float2 *>(part.ml + (slot * KV8_TC_ROWS + row) * 2) = make_float2(top, l);
                    }
                }
            }
        }
        tc_fence_before();
    }
    return true;
}

template <int DH>
__global__ void __launch_bounds__(TC_THREADS, 1) k_attention_kv8_tc(const AttnKV8Params p)
{
    extern __shared__ uint8_t smem_raw[];
    TcSmem<DH> &sm = *reinterpret_cast<TcSmem<DH> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5;
    wait_prior_grid();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sm.k_full[i]), 4);
            mbar_init(smem_addr(&sm.v_full[i]), 4);
            mbar_init(smem_addr(&sm.k_empty[i]), 1);
            mbar_init(smem_addr(&sm.v_empty[i]), 1);
            mbar_init(smem_addr(&sm.q_full[i]), 4);
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
        more_registers<152>();
        ok = softmax_role<DH>(p, sm, tmem, part);
    } else if (warp < 12) {
        fewer_registers<128>();
        ok = convert_role<DH>(p, sm, flags);
    } else {
        fewer_registers<80>();
        if (threadIdx.x == 12 * 32) {
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
