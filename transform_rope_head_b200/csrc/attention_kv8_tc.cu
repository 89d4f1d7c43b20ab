// Attention over the paged 8-bit cache on the 5th-generation tensor cores, for prompts and pieces of
// prompts (the mathematics and the work split: attention_kv8.cu).
//
// A unit is 256 query rows (tokens x heads of one key head) of a sequence, two M = 128 tiles that
// share every tile of 128 cached tokens.  Per tile of tokens and query tile
//   S [128 x 128] = Q K^T            tcgen05.mma kind::f16, both operands in shared memory
//   P = 2^(S c_j + log2 vs_j - m)    one thread per row, S read from tensor memory
//   O [128 x d_h] += P V             tcgen05.mma with P in tensor memory, over S's upper columns
// with fp32 accumulators.  The codes become 16-bit floats on their way to shared memory (exact: values fp16,
// keys the queries' type, so that queries need no conversion), rows of tokens for K and V alike in
// the 128-byte swizzle (V is read channels-major).
//
// Warps: 0-3 and 4-7 one query tile each (a thread a row: no exchange for maxima or sums), 8-11
// load and convert K and V two tiles ahead, 12 and 13 issue a query tile's MMAs each, S(i) | PV(i) S(i+1) | ...,
// so that the tensor cores work on one query tile while the other's exponentials are taken, 14 and 15
// fetch the next unit's queries.  A unit of at most 128 rows has one query tile; its tiles of tokens then go to
// the two in turn, as two streams of their own that are joined at its end, so that the MMAs of one still
// run beside the exponentials of the other.
//
// A row's thread reads S twice, for the maximum and for the exponentials, in chunks of 32 columns
// and rolled loops: the roles together have to fit the instruction caches (fully unrolled, their
// warps spent more time waiting for instructions than in any pipe).  A chunk is read and waited for in one
// place: between a tensor-memory load and its wait the compiler may not move its registers.
//
// The weights' offset moves only when a logit passes the largest one before by more than 2^8 (KV8_SLACK), so rescaling
// what was summed is rare.
//
// What bounds it: 4096 tokens behind 8192 (32 heads, d_h 128) take 817 to 841 us, 820 to 840
// TFLOP/s or 0.5 of cuBLAS' rate.
// Of a tile's 5000 cycles the tensor cores are busy 2050, the exponentials (16 a clock) 2050 and shared
// memory 3000; the two query tiles' softmax overlaps each other's MMAs, but a tile's own chain of S, maximum,
// P and PV is 3500 cycles long.  Tried: half rows on twice the warps 914 us (registers), 2^x of a quarter of
// the columns by polynomial +4%, polling waits +4%.  2048 tokens, d_h 64: 71 us, where units of few tiles pay
// for their beginning and end.
#include "attention_kv8.cuh"
#include "tcgen05.cuh"

namespace qkq {

namespace {

constexpr int TS = 128;            // cached tokens of a tile
constexpr int TC_THREADS = 16 * 32;
constexpr int CONV0 = 8 * 32;      // first converting thread
constexpr int MMA_WARP = 12;
constexpr int QUERY_WARP = 14;
constexpr int EXTRA = 3;           // what a unit costs besides its tiles, in tiles (1: 2 us more, 6: 5 us on 68)
constexpr int RING = 4;            // tiles whose steps are kept
constexpr int BLOCK = 128 * 128;   // bytes of 64 channels of 128 rows
template <int DH>
constexpr int QBUF = DH == 64 ? 2 : 1;  // units whose queries are held: what shared memory has room for

// Every row of a unit sees every token of the tile at tok0.
__device__ __forceinline__ bool all_visible(const AttnKV8Params &p, const KV8Span &span, int tok0)
{
    return tok0 + TS - 1 <= span.first && (p.window == 0 || tok0 > span.last - p.window || tok0 + TS - 1 < p.sinks);
}

// The units of a CTA's part, each warp on its own.  They live in shared memory: few of the fields are
// needed at a time, and registers are short.
struct Units {
    int64_t u0, hi;
    int b, qt, hk, j0, j1, number;
    KV8Seq s;
    KV8Span span;
    int rows;

    __device__ __forceinline__ void begin(const KV8Start &st)
    {
        u0 = st.u0;
        hi = st.hi;
        b = st.b;
        qt = st.qt;
        hk = st.hk;
        j0 = st.j0;
        number = 0;
    }
    __device__ __forceinline__ bool open(const AttnKV8Params &p)
    {
        if (u0 + EXTRA + j0 >= hi) return false;
        s = kv8_seq_checked(p.x, b);
        span = unit_span<TS>(p, s, qt, KV8_TC_ROWS);
        j1 = static_cast<int>(min(static_cast<int64_t>(span.count), hi - u0 - EXTRA));
        rows = min(KV8_TC_ROWS, s.n * p.ratio - qt * KV8_TC_ROWS);
        return true;
    }
    __device__ __forceinline__ void close(const AttnKV8Params &p)
    {
        ++number;
        if (j1 < span.count) {
            u0 = hi;
            return;
        }
        u0 += EXTRA + span.count;
        j0 = 0;
        if (u0 + EXTRA < hi) next_unit(p, s, KV8_TC_ROWS, b, qt, hk);
    }
    // A unit of one query tile: its token tiles go to the two query tiles' warps in turn.
    __device__ __forceinline__ bool narrow() const { return rows <= 128; }
    // Whether query tile t's warps have something of the unit.
    __device__ __forceinline__ bool has(int t) const { return !narrow() || t < j1 - j0; }
    __device__ __forceinline__ int token(int j) const { return TS * (j < span.head ? j : j + span.skip); }
    __device__ __forceinline__ bool full(const AttnKV8Params &p, int tok0) const { return all_visible(p, span, tok0); }
};

// The warp's first unit, or (after = true) its next one; false when there is none.
__device__ __forceinline__ bool take_unit(const AttnKV8Params &p, const KV8Start &st, Units &shared, bool after)
{
    Units u;
    if (after) {
        u = shared;
        u.close(p);
    } else {
        u.begin(st);
    }
    const bool more = u.open(p);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) shared = u;
    __syncwarp();
    return more;
}

template <int DH>
struct __align__(1024) TcSmem {
    uint8_t k[2][DH / 64][BLOCK];
    uint8_t v[2][DH / 64][BLOCK];
    uint8_t q[QBUF<DH>][2][DH / 64][BLOCK];
    // per 16 tokens: what a product is times to be a base-2 logit (above 0, so that -inf stays -inf), log2 and inverse
    // of the value step
    float4 step[RING][8];
    int2 tile[RING];                                // first token; whether every row sees all of the tile
    float2 stats[2][128];                           // (maximum, sum) of a narrow unit's two streams
    int nan_unit[4];                                // number + 1 of the unit whose masked tiles hold NaN values
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t q_full[QBUF<DH>][2], q_empty[QBUF<DH>][2], s_full[2], p_half[2], p_full[2], o_done[2], streams[4], drain, never;
    uint32_t tmem;
    KV8Start start;
    Units units[TC_THREADS / 32];
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

// A bounded wait by whole warps: the lanes go on, or give up, together.  The warp sleeps in the wait (up to
// 20 us a try): polling without the hint took a fifth of the kernel's issue slots.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned long long limit_ns)
{
    unsigned long long t0 = 0;
    for (;;) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity)
                     : "memory");
        if (__any_sync(FULL_MASK, ok)) return true;
        const unsigned long long t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (__any_sync(FULL_MASK, t - t0 > limit_ns)) return false;
    }
}
__device__ __forceinline__ bool warp_wait(const AttnKV8Params &p, uint32_t bar, uint32_t parity)
{
    return warp_wait(bar, parity, p.wait_limit_ns);
}

// Registers per thread of the warpgroups, 128 at launch: 2 x 136 + 144 + 96 = 4 x 128.
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

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

// Each warp converts 32 tokens of a tile, two slices of 16.
template <int DH>
__device__ __forceinline__ bool convert_role(const AttnKV8Params &p, TcSmem<DH> &sm, int &flags)
{
    constexpr int LPR = DH / 16;       // lanes per row
    constexpr int IT = LPR;            // rows per thread, RPI apart
    constexpr int RPI = 32 / LPR;
    const int tid = threadIdx.x - CONV0, lane = tid & 31, warp = tid >> 5;
    const int kc = lane % LPR, kr = lane / LPR;
    const uint32_t in_slice = kr * DH + 16 * kc;  // the thread's bytes from a slice's beginning on
    // where its rows' two pieces go; with 4 rows at a time every other row has another swizzle
    const uint32_t dst0 = row_offset<DH>(32 * warp + kr, 2 * kc), dst1 = row_offset<DH>(32 * warp + kr, 2 * kc + 1);
    // keys take the queries' type and the sign of the softmax scale, so that a logit grows with its product
    const uint32_t flip = p.scale_log2 < 0.0f ? 0x80808080u : 0u;
    int n = 0;  // tiles so far
    Units u;
    uint4 kw[IT], vw[IT];
    float ks = 0.0f, vs = 0.0f;     // lanes 0, 1: the steps of the warp's slices
    int id = -1;                    // in lanes 0, 1: their pages in the tile to be loaded next, as the table has them
    const uint8_t *k_at[2], *v_at[2];
    uint32_t none = 0;              // which of them have no page (nothing cached there, or a bad page)

    auto page_id = [&](int j) {
        const int tok = u.token(j) + 32 * warp + 16 * (lane & 1);
        return j < u.j1 && tok < u.s.len ? __ldg(p.x.block_table + static_cast<int64_t>(u.b) * p.x.max_pages + (tok >> p.x.page_shift)) : -1;
    };
    // tile j's slices, from the page ids (loaded before)
    auto locate = [&](int j) {
        const int tok = u.token(j) + 32 * warp + 16 * (lane & 1);
        const bool ok = id >= 0 && id < p.x.num_pages;
        if (!ok && tok < u.s.len) flags |= ST_CACHE_INDEX;
        none = __ballot_sync(FULL_MASK, !ok) & 3u;
        const int64_t ph = static_cast<int64_t>(ok ? id : 0) * p.Hkv + u.hk;
        const int64_t at = ((ph << p.x.page_shift) + (tok & ((1 << p.x.page_shift) - 1))) * DH;
        if (lane < 2) {
            ks = __ldg(p.k_steps + ph);
            vs = __ldg(p.v_steps + ph);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t slice = __shfl_sync(FULL_MASK, at, i) + in_slice;
            k_at[i] = p.k_codes + slice;
            v_at[i] = p.v_codes + slice;
        }
    };
    auto load = [&](uint4 (&w)[IT], const uint8_t *const (&at)[2]) {
#pragma unroll
        for (int i = 0; i < IT; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(at[i / (IT / 2)] + (i % (IT / 2)) * RPI * DH));
    };
    // rows of slices that `gone` names, and rows from `end` on, become zero
    auto clear = [&](uint4 (&w)[IT], uint32_t gone, int end) {
#pragma unroll
        for (int i = 0; i < IT; ++i)
            if (((gone >> (i / (IT / 2))) & 1) || 32 * warp + kr + i * RPI >= end) w[i] = make_uint4(0, 0, 0, 0);
    };
    auto store = [&](uint8_t *dst, const uint4 (&w)[IT], uint32_t signs, bool bf16) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const uint32_t x[4] = {w[i].x ^ signs, w[i].y ^ signs, w[i].z ^ signs, w[i].w ^ signs};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[2 * k] = e4m3x2_to_half2(x[k] & 0xffffu);
                h[2 * k + 1] = e4m3x2_to_half2(x[k] >> 16);
            }
            if (bf16) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h[k]));
                    h[k] = pack_bf16x2(v.x, v.y);
                }
            }
            const uint32_t turn = (i * RPI & 7) << 4;
            *reinterpret_cast<uint4 *>(dst + (dst0 ^ turn) + i * RPI * 128) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(dst + (dst1 ^ turn) + i * RPI * 128) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
    };

    if (static_cast<int>(blockIdx.x) == p.stalled_cta && !warp_wait(p, smem_addr(&sm.never), 0)) return false;
    u.begin(sm.start);
    bool more = u.open(p);
    int j = u.j0;
    if (more) {
        id = page_id(j);
        locate(j);
        load(kw, k_at);
        load(vw, v_at);
        id = page_id(j + 1);
    }
    while (more) {
        const int st = n & 1;
        const uint32_t par = ((n >> 1) & 1) ^ 1;
        const int tok0 = u.token(j), end = u.s.len - tok0, number = u.number;
        const bool full = u.full(p, tok0);
        const uint32_t gone = none;
        if (!warp_wait(p, smem_addr(&sm.k_empty[st]), par)) return false;
        if (lane < 2) {
            const bool here = !((gone >> lane) & 1);
            const float k1 = fminf(fmaxf(ks, KV8_STEP_MIN), KV8_STEP_MAX), v1 = fminf(fmaxf(vs, KV8_STEP_MIN), KV8_STEP_MAX);
            sm.step[n % RING][2 * warp + lane] = make_float4(fmaxf(here ? k1 * fabsf(p.scale_log2) : 0.0f, 1.17549435e-38f), here ? lg2(v1) : -INFINITY, here ? 1.0f / v1 : 0.0f, 0.0f);
            if (tid == 0) sm.tile[n % RING] = make_int2(tok0, full);
        }
        if (gone) clear(kw, gone, 128);
        if (p.half)
            store(&sm.k[st][0][0], kw, flip, false);
        else
            store(&sm.k[st][0][0], kw, flip, true);
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
            load(kw, k_at);
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
        if (!warp_wait(p, smem_addr(&sm.v_empty[st]), par)) return false;
        store(&sm.v[st][0][0], vw, 0u, false);
        if (lane == 0) mbar_arrive(smem_addr(&sm.v_full[st]));
        if (more) load(vw, v_at);
        ++n;
    }
    return true;
}

// Query tile t of each unit (of a narrow one, the only one), as it is, into the swizzled rows; rows that the
// unit has not become zero.
template <int DH>
__device__ __forceinline__ bool query_role(const AttnKV8Params &p, TcSmem<DH> &sm, int t)
{
    constexpr int LPR = DH / 8, RPI = 32 / LPR;
    const int lane = threadIdx.x & 31, c8 = lane % LPR, rl = lane / LPR;
    uint32_t phase = 0;  // bit buf: parity of that place's turn
    Units &u = sm.units[threadIdx.x >> 5];
    for (bool more = take_unit(p, sm.start, u, false); more; more = take_unit(p, sm.start, u, true)) {
        if (!u.has(t)) continue;
        const int buf = u.number % QBUF<DH>, skip = u.narrow() ? 0 : t * 128, rows = min(128, u.rows - skip);
        const int rr0 = u.qt * KV8_TC_ROWS + skip, token0 = p.div_ratio(rr0);
        const uint16_t *src = p.q + (static_cast<int64_t>(u.s.q0 + token0) * p.Hq + u.hk * p.ratio + rr0 - token0 * p.ratio) * DH + 8 * c8;
        const uint32_t dst = smem_addr(&sm.q[buf][t][0][0]);
        if (!warp_wait(p, smem_addr(&sm.q_empty[buf][t]), ((phase >> buf) & 1) ^ 1)) return false;
        phase ^= 1u << buf;
#pragma unroll 2
        for (int r8 = 0; r8 < 128; r8 += 8) {
#pragma unroll
            for (int i = 0; i < 8; i += RPI) {
                const int r = r8 + i + rl;
                // at most 128 tokens of 2^16 heads on: 32 bits
                const bool in = r < rows;
                const uint32_t off = in ? static_cast<uint32_t>(r + (p.div_ratio(rr0 + r) - token0) * (p.Hq - p.ratio)) * DH : 0u;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + r8 * 128 + row_offset<DH>(i + rl, c8)), "l"(src + off), "r"(in ? 16 : 0)
                             : "memory");
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.q_full[buf][t]));
    }
    return true;
}

// The MMAs of query tile t, tile by tile: the tile before's values, then the tile's scores (which take the
// columns that P leaves).  Both MMA warps take part in every token tile, in order: what the other one computes (of a
// narrow unit) a warp waits for and lets go.  A wait tells a barrier's phase from its neighbours only, so a warp
// that passed over tiles could take an older phase for the one it means.
template <int DH>
__device__ __forceinline__ bool mma_role(const AttnKV8Params &p, TcSmem<DH> &sm, uint32_t tmem, int t)
{
    const uint32_t id_s = p.half ? idesc_f16(TS) : idesc_bf16(TS), id_o = idesc_f16(DH) | (1u << 16);  // V: channels-major
    // K, Q: rows of 64 channels, 8-row groups 1024 bytes apart; V: 64 channels of a token a row, 8-token
    // groups 1024 bytes, 64-channel blocks BLOCK bytes apart
    constexpr uint64_t STAGE = (DH / 64) * (BLOCK >> 4);
    const uint64_t k0 = sw128_desc(smem_addr(&sm.k[0][0][0]));
    const uint64_t v0 = (sw128_desc(smem_addr(&sm.v[0][0][0])) & ~(0x3fffull << 16)) | (static_cast<uint64_t>(BLOCK >> 4) << 16);
    const uint32_t s_cols = tmem + t * TS, o_cols = tmem + 2 * TS + t * DH;
    int n = 0;
    uint32_t q_phase = 0, p_phase = 0;  // parities: bit buf; bit 0
    // tile i's keys or values, which the other warp reads
    auto let_go = [&](uint64_t (&full)[2], uint64_t (&empty)[2], int i) {
        if (!warp_wait(p, smem_addr(&full[i & 1]), (i >> 1) & 1)) return false;
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&empty[i & 1]));
        return true;
    };
    Units &u = sm.units[threadIdx.x >> 5];
    for (bool more = take_unit(p, sm.start, u, false); more; more = take_unit(p, sm.start, u, true)) {
        const int tiles = u.j1 - u.j0, buf = u.number % QBUF<DH>;
        // its tiles: all, or of a narrow unit every other one
        const bool narrow = u.narrow();
        const int first = narrow ? t : 0, step = narrow ? 2 : 1, count = narrow ? (tiles + 1 - t) / 2 : tiles;
        if (!u.has(t)) {
            for (int i = n; i < n + tiles; ++i)
                if (!let_go(sm.k_full, sm.k_empty, i) || !let_go(sm.v_full, sm.v_empty, i)) return false;
            n += tiles;
            continue;
        }
        const uint64_t q = sw128_desc(smem_addr(&sm.q[buf][t][0][0]));
        if (!warp_wait(p, smem_addr(&sm.q_full[buf][t]), (q_phase >> buf) & 1)) return false;
        q_phase ^= 1u << buf;
        if (first > 0 && (!let_go(sm.k_full, sm.k_empty, n) || !let_go(sm.v_full, sm.v_empty, n))) return false;
#pragma unroll 1
        for (int k = 0; k <= count; ++k) {
            if (k > 0) {
                const int i = n + first + (k - 1) * step, st = i & 1;
                const uint64_t v = v0 + st * STAGE;
                const uint32_t add = k > 1 ? 1u : 0u;
                if (!warp_wait(p, smem_addr(&sm.v_full[st]), (i >> 1) & 1)) return false;
                if (!warp_wait(p, smem_addr(&sm.p_half[t]), p_phase)) return false;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int s = TS / 32; s < TS / 16; ++s)
                        mma_f16_ts(o_cols, s_cols + TS / 2 + 8 * s, v + s * (16 * 128 >> 4), id_o, s > TS / 32 ? 1u : add);
                }
                __syncwarp();
                if (!warp_wait(p, smem_addr(&sm.p_full[t]), p_phase)) return false;
                p_phase ^= 1u;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < TS / 32; ++s) mma_f16_ts(o_cols, s_cols + TS / 2 + 8 * s, v + s * (16 * 128 >> 4), id_o, 1u);
                    mma_commit(smem_addr(&sm.v_empty[st]));
                    if (k == count) mma_commit(smem_addr(&sm.o_done[t]));
                }
                __syncwarp();
                if (narrow && i + 1 < n + tiles && !let_go(sm.v_full, sm.v_empty, i + 1)) return false;
            }
            if (k < count) {
                const int i = n + first + k * step, st = i & 1;
                const uint64_t kd = k0 + st * STAGE;
                if (!warp_wait(p, smem_addr(&sm.k_full[st]), (i >> 1) & 1)) return false;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < DH / 16; ++s) {
                        const uint32_t off = ((s >> 2) * BLOCK + (s & 3) * 32) >> 4;
                        mma_bf16(s_cols, q + off, kd + off, id_s, s ? 1u : 0u);
                    }
                    // done when all before it is, the last tile's values among that
                    mma_commit(smem_addr(&sm.s_full[t]));
                    mma_commit(smem_addr(&sm.k_empty[st]));
                    if (k + 1 == count) mma_commit(smem_addr(&sm.q_empty[buf][t]));
                }
                __syncwarp();
                // before this tile's softmax is waited for, so that the other stream's next keys can come
                if (narrow && i + 1 < n + tiles && !let_go(sm.k_full, sm.k_empty, i + 1)) return false;
            }
        }
        n += tiles;
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

// Columns that the row does not see become -inf.
__device__ __forceinline__ void hide(uint32_t (&raw)[32], uint32_t bits)
{
#pragma unroll
    for (int i = 0; i < 32; ++i) raw[i] = (bits >> i) & 1 ? raw[i] : 0xff800000u;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The largest base-2 logit (without the maximum's offset) of 32 columns.
__device__ __forceinline__ float chunk_top(const uint32_t (&raw)[32], const float4 *step)
{
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        float x[2] = {__uint_as_float(raw[16 * g]), __uint_as_float(raw[16 * g + 1])};
#pragma unroll
        for (int i = 2; i < 16; i += 4) {
            x[0] = max3(x[0], __uint_as_float(raw[16 * g + i]), __uint_as_float(raw[16 * g + i + 1]));
            if (i + 2 < 16) x[1] = max3(x[1], __uint_as_float(raw[16 * g + i + 2]), __uint_as_float(raw[16 * g + i + 3]));
        }
        // the factor is positive and rounding keeps order: the logit of the maximum
        top = fmaxf(top, __fmaf_rn(fmaxf(x[0], x[1]), step[g].x, step[g].y));
    }
    return top;
}

// P of 32 columns as fp16 pairs, and their part of the row's sum.
__device__ __forceinline__ void chunk_p(const uint32_t (&raw)[32], const float4 &step0, const float4 &step1, float m,
                                        uint32_t (&pw)[16], float &l)
{
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const float4 &step = g ? step1 : step0;
        const float f = step.x, a = step.y - m;
        const uint64_t f2 = pair(f, f), a2 = pair(a, a);
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = 16 * g + 2 * i;
            float x, y;
            unpair(fma_pair(pair(__uint_as_float(raw[k]), __uint_as_float(raw[k + 1])), f2, a2), x, y);
            x = ex2(x);
            y = ex2(y);
            sum = add_pair(sum, pair(x, y));
            pw[8 * g + i] = pack_weights(x, y);
        }
        float x, y;
        unpair(sum, x, y);
        l = __fmaf_rn(x + y, step.z, l);
    }
}

// A row's statistics: m the weights' offset, l the sum, pass what a logit must
// exceed to move m (-inf: none seen yet).
struct RowState {
    float m, l, pass;
};

// S of one tile to P, the row's thread.  (Tiles that every row sees whole have code of their own: with the
// masking in it, skipped as it was, the same loop took a fifth longer.)
template <int DH, bool MASKED>
__device__ __forceinline__ void softmax_tile(const float4 *step, uint32_t p_half, uint32_t p_full, bool first, uint32_t s_cols,
                                             uint32_t o_cols, const RowMask &mask, RowState &r)
{
    uint32_t a[32], b[32], pw[16];
    float top = -INFINITY;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        tmem_ld32_async(s_cols + 64 * h, a);
        tmem_ld32_async(s_cols + 64 * h + 32, b);
        tmem_ld_wait(a);
        tmem_ld_wait(b);
        if (MASKED) {
            hide(a, mask.bits(64 * h));
            hide(b, mask.bits(64 * h + 32));
        }
        top = fmaxf(top, chunk_top(a, step + 4 * h));
        top = fmaxf(top, chunk_top(b, step + 4 * h + 2));
    }
    const bool moves = top > r.pass;
    if (__any_sync(FULL_MASK, moves)) {
        // the maximum moves (before a row's first logit there is nothing to rescale)
        const float to = moves ? top - KV8_UP : r.m;
        const float alpha = !moves ? 1.0f : r.pass > -INFINITY ? ex2(r.m - to) : 0.0f;
        if (moves) {
            r.m = to;
            r.pass = top + KV8_SLACK;
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
#pragma unroll 1
    for (int h = 1; h >= 0; --h) {
        tmem_ld32_async(s_cols + 64 * h, a);
        tmem_ld32_async(s_cols + 64 * h + 32, b);
        const float4 c0 = step[4 * h], c1 = step[4 * h + 1], c2 = step[4 * h + 2], c3 = step[4 * h + 3];
        tmem_ld_wait(a);
        tmem_ld_wait(b);
        if (MASKED) {
            hide(a, mask.bits(64 * h));
            hide(b, mask.bits(64 * h + 32));
        }
        chunk_p(b, c2, c3, r.m, pw, r.l);
        tmem_st16(s_cols + TS / 2 + 32 * h + 16, pw);
        chunk_p(a, c0, c1, r.m, pw, r.l);
        tmem_st16(s_cols + TS / 2 + 32 * h, pw);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(h ? p_half : p_full);
    }
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
    int n = 0, cnt = 0;        // tiles of the part, and of them this query tile's
    uint32_t done[2] = {0, 0}; // parities of the query tiles' units
    uint32_t met = 0;
    // the two warps that have the same rows of the query tiles
    auto meet = [&]() {
        const uint32_t bar = smem_addr(&sm.streams[r >> 5]);
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
        met ^= 1u;
        return warp_wait(p, bar, met ^ 1u);
    };
    Units &u = sm.units[threadIdx.x >> 5];
    for (bool more = take_unit(p, sm.start, u, false); more; more = take_unit(p, sm.start, u, true)) {
        const int tiles = u.j1 - u.j0;
        const bool narrow = u.narrow(), two = narrow && tiles > 1;
        const uint32_t done0 = done[0], done1 = done[1];
        done[0] ^= 1u;
        if (u.has(1)) {
            done[1] ^= 1u;
        } else if (!meet()) {  // the second tile's warps have ended what they had before the first's go on alone
            return false;
        }
        if (!u.has(t)) {
            n += tiles;
            continue;
        }
        const int row = narrow ? r : t * 128 + r, step = narrow ? 2 : 1;
        const bool live = row < u.rows;
        const int at = live ? u.s.len - u.s.n + p.div_ratio(u.qt * KV8_TC_ROWS + row) : -1;
        RowState st{0.0f, 0.0f, -INFINITY};
        const int last = n + tiles;
        bool first = true;
#pragma unroll 1
        for (int i = narrow ? n + t : n; i < last; i += step, ++cnt) {
            if (!warp_wait(p, smem_addr(&sm.s_full[t]), cnt & 1)) return false;
            tc_fence_after();
            const int2 tile = sm.tile[i % RING];
            const int hi = at - tile.x + 1;
            const RowMask mask{hi, p.window ? hi - p.window : 0, p.window ? p.sinks - tile.x : 0};
            const uint32_t p_half = smem_addr(&sm.p_half[t]), p_full = smem_addr(&sm.p_full[t]);
            if (tile.y)
                softmax_tile<DH, false>(sm.step[i % RING], p_half, p_full, first, s_cols, o_cols, mask, st);
            else
                softmax_tile<DH, true>(sm.step[i % RING], p_half, p_full, first, s_cols, o_cols, mask, st);
            first = false;
        }
        n = last;

        // ---- the unit's end ------------------------------------------------------------------------
        if (!warp_wait(p, smem_addr(&sm.o_done[t]), t ? done1 : done0)) return false;
        float top = st.pass == -INFINITY ? -INFINITY : st.m, f0 = 1.0f, f1 = 0.0f;
        if (two) {
            // the other stream's sums stand in the same lanes: each of a row's two threads joins half of the channels
            sm.stats[t][r] = make_float2(top, st.l);
            if (!meet()) return false;
            // complete by now (and its next turn is not): only the order of what was written is left to wait for
            if (!warp_wait(p, smem_addr(&sm.o_done[t ^ 1]), t ? done0 : done1)) return false;
            const float2 a = sm.stats[0][r], b = sm.stats[1][r];
            top = fmaxf(a.x, b.x);
            f0 = a.x == -INFINITY ? 0.0f : ex2(a.x - top);
            f1 = b.x == -INFINITY ? 0.0f : ex2(b.x - top);
            st.l = __fmaf_rn(b.y, f1, a.y * f0);
        }
        tc_fence_after();
        const bool whole = u.j0 == 0 && u.j1 == u.span.count;
        const bool nan = *reinterpret_cast<volatile int *>(&sm.nan_unit[u.number & 3]) == u.number + 1;
        const bool empty = top == -INFINITY && st.l == 0.0f;
        const int rr = u.qt * KV8_TC_ROWS + row, token = p.div_ratio(rr);
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (u.number == 0 ? 0 : 1);
        const int64_t q_row = static_cast<int64_t>(u.s.q0) * p.Hq + u.hk * p.ratio + rr + static_cast<int64_t>(token) * (p.Hq - p.ratio);
        const float inv = empty ? 0.0f : 1.0f / st.l;
#pragma unroll 1
        for (int c = two ? t * (DH / 2) : 0; c < (two && t == 0 ? DH / 2 : DH); c += 16) {
            uint32_t raw[16];
            __syncwarp();
            if (two) {
                uint32_t other[16];
                tmem_ld16(lanes + 2 * TS + c, raw);
                tmem_ld16(lanes + 2 * TS + DH + c, other);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    raw[i] = __float_as_uint(__fmaf_rn(__uint_as_float(other[i]), f1, __uint_as_float(raw[i]) * f0));
            } else {
                tmem_ld16(o_cols + c, raw);
            }
            if (!live) continue;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
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
        if (live && !(two && t == 1)) {
            if (!whole)
                *reinterpret_cast<float2 *>(part.ml + (slot * KV8_TC_ROWS + row) * 2) = make_float2(top, st.l);
            else if (p.lse)
                p.lse[q_row] = empty ? -INFINITY : (lg2(st.l) + top) * 0.6931471805599453f;
        }
        tc_fence_before();
        if (two) {
            // neither goes on to write O while the other reads it
            if (!meet()) return false;
            tc_fence_after();
        }
    }
    return true;
}

// A wait of this CTA gave up: what its part was to give, its units' rows or their partial statistics, becomes NaN, so
// that a caller who does not look at the status cannot take what stood there for results.  By the warps that have
// kept the registers a called function may use.
template <int DH>
__device__ __noinline__ void void_part(const AttnKV8Params &p, const KV8Start &start)
{
    const KV8Partials part(p.workspace, gridDim.x, KV8_TC_ROWS, DH);
    constexpr float NOT = __builtin_nanf("");
    const uint32_t w = pack16(NOT, NOT, p.half);
    Units u;
    u.begin(start);
    while (u.open(p)) {
        const bool whole = u.j0 == 0 && u.j1 == u.span.count;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (u.number == 0 ? 0 : 1);
        for (int i = threadIdx.x; i < u.rows * (DH / 8); i += MMA_WARP * 32) {
            const int row = i / (DH / 8), c = i % (DH / 8), rr = u.qt * KV8_TC_ROWS + row;
            const int64_t q_row = static_cast<int64_t>(u.s.q0) * p.Hq + u.hk * p.ratio + rr + static_cast<int64_t>(p.div_ratio(rr)) * (p.Hq - p.ratio);
            if (whole) *reinterpret_cast<uint4 *>(p.out + q_row * DH + 8 * c) = make_uint4(w, w, w, w);
            if (whole && c == 0 && p.lse) p.lse[q_row] = NOT;
            if (!whole && c == 0) *reinterpret_cast<float2 *>(part.ml + (slot * KV8_TC_ROWS + row) * 2) = make_float2(0.0f, NOT);
        }
        u.close(p);
    }
}

template <int DH>
__global__ void __launch_bounds__(TC_THREADS, 1) k_attention_kv8_tc(const __grid_constant__ AttnKV8Params p)
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
            mbar_init(smem_addr(&sm.k_empty[i]), 2);
            mbar_init(smem_addr(&sm.v_empty[i]), 2);
#pragma unroll
            for (int b = 0; b < QBUF<DH>; ++b) {
                mbar_init(smem_addr(&sm.q_full[b][i]), 1);
                mbar_init(smem_addr(&sm.q_empty[b][i]), 1);
            }
            mbar_init(smem_addr(&sm.s_full[i]), 1);
            mbar_init(smem_addr(&sm.p_half[i]), 4);
            mbar_init(smem_addr(&sm.p_full[i]), 4);
            mbar_init(smem_addr(&sm.o_done[i]), 1);
            mbar_init(smem_addr(&sm.streams[2 * i]), 2);
            mbar_init(smem_addr(&sm.streams[2 * i + 1]), 2);
        }
        mbar_init(smem_addr(&sm.drain), 2);
        mbar_init(smem_addr(&sm.never), 1);  // nothing arrives
        fence_mbar_init();
#pragma unroll
        for (int i = 0; i < 4; ++i) sm.nan_unit[i] = 0;
    }
    if (warp == MMA_WARP) {
        tmem_alloc(smem_addr(&sm.tmem), 512);
        tmem_relinquish();
    }
    find_start<TS, KV8_TC_ROWS, TC_THREADS>(p, sm.start, EXTRA, 1);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    allow_next_grid();  // after the allocation: a later grid's must not come first
    const uint32_t tmem = sm.tmem;
    const KV8Partials part(p.workspace, gridDim.x, KV8_TC_ROWS, DH);
    if (threadIdx.x == 0)
        part.meta[blockIdx.x] = KV8Meta{sm.start.u0, sm.start.j0, sm.start.b, sm.start.qt, sm.start.hk};

    int flags = threadIdx.x == 0 ? sm.start.flags : 0;
    bool ok = true;
    if (warp < 8) {
        more_registers<136>();
        ok = softmax_role<DH>(p, sm, tmem, part);
    } else if (warp < MMA_WARP) {
        more_registers<144>();
        ok = convert_role<DH>(p, sm, flags);
    } else {
        fewer_registers<96>();
        if (warp >= QUERY_WARP) {
            ok = query_role<DH>(p, sm, warp - QUERY_WARP);
        } else {
            ok = mma_role<DH>(p, sm, tmem, warp - MMA_WARP);
            // nothing of this CTA runs on when its tensor memory goes
            if (elect_one()) mma_commit(smem_addr(&sm.drain));
            __syncwarp();
            ok &= warp_wait(smem_addr(&sm.drain), 0, WAIT_LIMIT_NS);
        }
        __syncwarp();
    }
    if (!ok) flags |= ST_TIMEOUT;
    if (p.status && flags) atomicOr(p.status, flags);
    __syncwarp();
    tc_fence_before();
    const bool gave_up = __syncthreads_or(!ok);
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (gave_up && warp < MMA_WARP) void_part<DH>(p, sm.start);
}

// The waits of a test: their limit, and the CTA whose first tile never comes.
std::atomic<unsigned long long> wait_limit{WAIT_LIMIT_NS};
std::atomic<int> stalled_cta{-1};

template <int DH>
cudaError_t launch(const AttnKV8Params &p, const DeviceInfo &dev, cudaStream_t stream)
{
    constexpr int smem = sizeof(TcSmem<DH>) + 1024;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(allowed, k_attention_kv8_tc<DH>, smem, dev.ordinal);
    if (e != cudaSuccess) return e;
    const int ctas = dev.num_sms < KV8_TC_MAX_CTAS ? dev.num_sms : KV8_TC_MAX_CTAS;
    const cudaError_t f = launch_after_prior(k_attention_kv8_tc<DH>, dim3(ctas), dim3(TC_THREADS), smem, stream, p);
    if (f != cudaSuccess) return f;
    return attention_kv8_join_launch(p, DH, ctas, KV8_TC_ROWS, stream);
}

}  // namespace

void attention_kv8_stall(unsigned long long limit_ns, int cta)
{
    wait_limit.store(limit_ns ? limit_ns : WAIT_LIMIT_NS, std::memory_order_relaxed);
    stalled_cta.store(limit_ns ? cta : -1, std::memory_order_relaxed);
}

cudaError_t attention_kv8_tc_launch(const AttnKV8Params &params, int d_h, const DeviceInfo &dev, cudaStream_t stream)
{
    AttnKV8Params p = params;
    p.wait_limit_ns = wait_limit.load(std::memory_order_relaxed);
    p.stalled_cta = stalled_cta.load(std::memory_order_relaxed);
    const cudaError_t e = d_h == 64 ? launch<64>(p, dev, stream) : launch<128>(p, dev, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qkq
