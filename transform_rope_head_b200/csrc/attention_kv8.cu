// Attention over the paged 8-bit cache for few query rows per sequence: one decoding token, a
// handful of drafted ones.
//
// out[t][h] = sum_j p_j vs_j vc_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = scale log2(e) ks_j (q . kc_j)
// over the cached tokens j that query t may see (j <= its index; with a window W also
// j > index - W or j < sinks); kc, vc the e4m3 codes, ks, vs their page's steps.
//
// Memory bound: the codes of every visible cached token are read once, 2 d_h bytes per key head.
// Each warp takes slices of 16 cached tokens of one key head against up to 8 NT query rows
// (tokens x heads of the key head), the products as warp-level fp16 MMAs (m16n8k16, fp32 sums)
// with the cached tokens on the wide side, so a decoding step's few rows waste little:
//   S^T [16 tokens x rows]  = K [16 x d_h] Q^T,   O^T [d_h x rows] += V^T [d_h x 16] P^T.
// Codes come by cp.async into a ring of two slices per warp in shared memory and go from there straight
// into the A fragments: a lane's 16-byte reads hold the channels (K) or channel x token pairs (V) that
// its fragment needs, which channel stands at which index being free as long as both operands
// agree; e4m3 -> fp16 is one exact conversion per pair.  (Held in registers on their way, a slice
// more of 32 registers a lane or 12 warps an SM: 64 sequences x 8192 tokens 136 us; the ring 107 us, 5.5 TB/s
// or 0.84 of the copy rate; three slices as fast, four leave too few warps: 178 us.)
// Queries are scaled by a power of two per row into fp16's range (bf16's 8 bits fit its 11).  P is
// rounded to fp16 (relative 2^-12 mean); sums, maxima and the output stay fp32.  The page's value step
// goes into the exponent, w_j = p_j vs_j = 2^(s_j + log2 vs_j - m), so that m bounds what is
// rounded, and the row sum takes w_j / vs_j.  m moves only when a logit passes the largest one before by
// more than 2^8 (KV8_SLACK), which leaves most slices without any exchange.
//
// Work split: the slices of all (sequence, query block, key head) in one line, each unit with 12 places
// more for what beginning and ending it costs, cut into equal parts, one per CTA of a persistent grid,
// found from the lengths on the device: ragged batches balance without the host knowing a length.  What a
// part shares with its neighbours goes to the workspace as (rows, maximum, sum) and a second kernel joins
// it in a fixed order.  One token x 131072: 54 us, 5.0 TB/s, of which 35 us the slices; the rest is the start
// (2 us), the first pages and queries, the parts' join and two launches.
#include "attention_kv8.cuh"

namespace qkq {

namespace {

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

constexpr int EXTRA = 12;  // what a unit costs besides its slices, in slices
constexpr int RING = 2;    // slices of a warp in use and on their way (3: as fast, 4: fewer warps fit)

// A warp's slices on their way: codes by cp.async (what is in flight costs no registers), K rows then V rows.
// 16-byte pieces of a row (of two rows of 64 channels) stand XORed among the 128 bytes' eight places so that
// the fragments' reads meet no bank twice: K reads 4 neighbours of two rows at a time, V one piece
// of every other row.
template <int DH>
struct __align__(128) Ring {
    uint8_t codes[RING][2][16 * DH];
    float ks[RING], vs[RING];
    int page[RING];
};

template <int DH>
__device__ __forceinline__ uint32_t piece(int row, int c)
{
    if (DH == 128) return row * 128 + ((c ^ (row & 6) ^ ((row & 1) << 2)) << 4);
    return (row >> 1) * 128 + ((((row & 1) * 4 + c) ^ (((row >> 1) & 3) << 1)) << 4);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Starts the copies of the slice at tok0 (none without a page).
template <int DH>
__device__ __forceinline__ void start_slice(Ring<DH> &ring, int st, const AttnKV8Params &p, int page, int hk, int tok0, int lane)
{
    constexpr int PER_ROW = DH / 16, RPI = 32 / PER_ROW;
    if (lane == 0) ring.page[st] = page;
    const int64_t ph = static_cast<int64_t>(page < 0 ? 0 : page) * p.Hkv + hk;
    const int64_t base = ((ph << p.x.page_shift) + (tok0 & ((1 << p.x.page_shift) - 1))) * DH + 16 * lane;
    const int r = lane / PER_ROW, c = lane % PER_ROW;
#pragma unroll
    for (int i = 0; i < 16; i += RPI) {
        copy16(smem_addr(ring.codes[st][0]) + piece<DH>(r + i, c), p.k_codes + base + i * DH);
        copy16(smem_addr(ring.codes[st][1]) + piece<DH>(r + i, c), p.v_codes + base + i * DH);
    }
    if (lane == 0) copy4(smem_addr(&ring.ks[st]), p.k_steps + ph);
    if (lane == 1) copy4(smem_addr(&ring.vs[st]), p.v_steps + ph);
}

// One slice's codes and steps as this lane holds them.
template <int DH>
struct Slice {
    uint32_t k[2][DH / 16];  // tokens g, g + 8: channels 16 t .. of each 64
    uint32_t v[4][DH / 32];  // tokens 2t, 2t + 1, 2t + 8, 2t + 9: channels g * DH / 8 ..
};

template <int DH>
__device__ __forceinline__ void read_slice(Slice<DH> &s, const Ring<DH> &ring, int st, int g, int t)
{
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < DH / 64; ++c) {
            const uint4 w = *reinterpret_cast<const uint4 *>(ring.codes[st][0] + piece<DH>(g + 8 * r, 4 * c + t));
            s.k[r][4 * c] = w.x;
            s.k[r][4 * c + 1] = w.y;
            s.k[r][4 * c + 2] = w.z;
            s.k[r][4 * c + 3] = w.w;
        }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = 2 * t + (r & 1) + 8 * (r >> 1);
        if (DH == 128) {
            const uint4 w = *reinterpret_cast<const uint4 *>(ring.codes[st][1] + piece<DH>(row, g));
            s.v[r][0] = w.x;
            s.v[r][1] = w.y;
            s.v[r][DH / 32 - 2] = w.z;
            s.v[r][DH / 32 - 1] = w.w;
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(ring.codes[st][1] + piece<DH>(row, g >> 1) + 8 * (g & 1));
            s.v[r][0] = w.x;
            s.v[r][1] = w.y;
        }
    }
}

template <int DH, int NT, int NW>
struct MergeSmem {
    float o[NW][8 * NT][DH];
    float m[NW][8 * NT], l[NW][8 * NT];
};

template <int DH, int NT, int NW>
__global__ void __launch_bounds__(NW * 32, NT == 1 ? 3 : 2) k_attention_kv8(const __grid_constant__ AttnKV8Params p)
{
    constexpr int R = 8 * NT;     // query rows of a unit
    constexpr int KS = DH / 16;   // K-steps of S, M tiles of O
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Ring<DH> *const rings = reinterpret_cast<Ring<DH> *>(smem_raw);
    MergeSmem<DH, NT, NW> &sm = *reinterpret_cast<MergeSmem<DH, NT, NW> *>(smem_raw + NW * sizeof(Ring<DH>));
    __shared__ KV8Start s_start;
    wait_prior_grid();
    allow_next_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const KV8Index &x = p.x;
    const KV8Partials part(p.workspace, gridDim.x, R, DH);

    find_start<16, R, NW * 32>(p, s_start, EXTRA, NW);  // at least a slice per warp
    int64_t u0 = s_start.u0;
    const int64_t hi = s_start.hi;
    int b = s_start.b, qt = s_start.qt, hk = s_start.hk;
    int j0 = s_start.j0;
    if (threadIdx.x == 0) part.meta[blockIdx.x] = KV8Meta{u0, j0, b, qt, hk};
    int flags = s_start.flags;
    bool first = true;

    while (u0 + EXTRA + j0 < hi) {
        const KV8Seq s = kv8_seq_checked(x, b);
        const KV8Span span = unit_span<16>(p, s, qt, R);
        const int j1 = static_cast<int>(min(static_cast<int64_t>(span.count), hi - u0 - EXTRA));
        const int rows = min(R, s.n * p.ratio - qt * R);

        // ---- the warp's first slices, on their way while the queries come ---------------------
        auto token = [&](int j) { return 16 * (j < span.head ? j : j + span.skip); };
        // pages as the table has them are checked when they are needed, not when they are asked for
        auto raw_page = [&](int j) {
            const int tok = token(j);
            return j < j1 && tok < s.len ? __ldg(x.block_table + static_cast<int64_t>(b) * x.max_pages + (tok >> x.page_shift)) : -1;
        };
        auto checked = [&](int j, int raw) {
            if (raw >= 0 && raw < x.num_pages) return raw;
            if (j < j1 && token(j) < s.len) flags |= ST_CACHE_INDEX;
            return -1;
        };
        Ring<DH> &ring = rings[warp];
        int j = j0 + warp, st = 0;
        int raw[RING];
#pragma unroll
        for (int i = 0; i < RING; ++i) raw[i] = raw_page(j + i * NW);
        uint4 qw[NT][DH / 32];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int rr = qt * R + 8 * n + g, tk = p.div_ratio(rr);
            const uint16_t *src = p.q + (static_cast<int64_t>(s.q0 + tk) * p.Hq + hk * p.ratio + rr - tk * p.ratio) * DH + 16 * t;
#pragma unroll
            for (int c = 0; c < DH / 32; ++c) {
                qw[n][c] = make_uint4(0, 0, 0, 0);
                if (8 * n + g < rows) qw[n][c] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * (c >> 1) + 8 * (c & 1)));
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < RING - 1; ++i) {
            const int ji = j + i * NW, page = checked(ji, raw[i]);
            if (ji < j1) start_slice<DH>(ring, i, p, page, hk, token(ji), lane);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        int raw_next = raw[RING - 1];

        // ---- this unit's queries: B fragments, scaled per row into fp16 --------------------
        uint32_t qf[NT][KS][2];
        float fac[NT][2];   // rows 2t, 2t + 1 of each n-tile: scale log2(e) / the row's factor
        int at[NT][2];      // their index in the sequence (none: -1)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = 8 * n + g;
            float2 v[KS][2];
            float amax = 0.0f;
#pragma unroll
            for (int c = 0; c < DH / 32; ++c) {
                const uint32_t u[4] = {qw[n][c].x, qw[n][c].y, qw[n][c].z, qw[n][c].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x2 = unpack16(u[e], p.half);
                    v[2 * c + (e >> 1)][e & 1] = x2;
                    amax = fmaxf(amax, fabsf(x2.x) <= 3.402823466e38f ? fabsf(x2.x) : 0.0f);
                    amax = fmaxf(amax, fabsf(x2.y) <= 3.402823466e38f ? fabsf(x2.y) : 0.0f);
                }
            }
            amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, 2));
            const int e = row_exponent(amax);
            const float up = exp2i(-e);
            const float f = p.scale_log2 * exp2i(e);
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) qf[n][k][h] = pack16(v[k][h].x * up, v[k][h].y * up, true);
            const int idx = row < rows ? s.len - s.n + p.div_ratio(qt * R + row) : -1;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                fac[n][c] = __shfl_sync(FULL_MASK, f, (2 * t + c) * 4);
                at[n][c] = __shfl_sync(FULL_MASK, idx, (2 * t + c) * 4);
            }
        }

        float o[NT][KS][4];
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][k][e] = 0.0f;
        }

        // ---- the warp's slices -------------------------------------------------------------
        for (; j < j1; j += NW) {
            // the copies RING - 1 slices on, into the place of the slice before
            const int ahead = j + (RING - 1) * NW;
            const int page_ahead = checked(ahead, raw_next);
            if (ahead < j1) start_slice<DH>(ring, st == 0 ? RING - 1 : st - 1, p, page_ahead, hk, token(ahead), lane);
            asm volatile("cp.async.commit_group;" ::: "memory");
            raw_next = raw_page(ahead + NW);
            asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
            __syncwarp();
            Slice<DH> sl;
            read_slice<DH>(sl, ring, st, g, t);
            const int page = ring.page[st];
            const float ks = fminf(fmaxf(ring.ks[st], KV8_STEP_MIN), KV8_STEP_MAX);
            const float vs = fminf(fmaxf(ring.vs[st], KV8_STEP_MIN), KV8_STEP_MAX);
            st = st == RING - 1 ? 0 : st + 1;
            const int tok0 = token(j);
            // two chains of sums, half as long
            float sc[NT][4], sd[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[n][e] = sd[n][e] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint32_t a0 = e4m3x2_to_half2(sl.k[0][k] & 0xffffu), a2 = e4m3x2_to_half2(sl.k[0][k] >> 16);
                const uint32_t a1 = e4m3x2_to_half2(sl.k[1][k] & 0xffffu), a3 = e4m3x2_to_half2(sl.k[1][k] >> 16);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(k & 1 ? sd[n] : sc[n], a0, a1, a2, a3, qf[n][k][0], qf[n][k][1]);
            }
            const float lvs = lg2(vs), ivs = 1.0f / vs;
            // every row sees every token of the slice?
            const bool full = page >= 0 && tok0 + 15 <= span.first &&
                              (p.window == 0 || tok0 > span.last - p.window || tok0 + 15 < p.sinks);
            bool passes = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sc[n][e] = __fmaf_rn(sc[n][e] + sd[n][e], fac[n][e & 1] * ks, lvs);
                    if (!full) {
                        const int tok = tok0 + g + 8 * (e >> 1);
                        const int i = at[n][e & 1];
                        const bool see = page >= 0 && tok <= i && (p.window == 0 || tok > i - p.window || tok < p.sinks);
                        if (!see) sc[n][e] = -INFINITY;
                    }
                    passes |= sc[n][e] > m[n][e & 1] + (KV8_UP + KV8_SLACK);
                }
            if (__any_sync(FULL_MASK, passes)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float top = fmaxf(sc[n][c], sc[n][2 + c]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, off));
                        top = fmaxf(top - KV8_UP, m[n][c]);
                        const float alpha = m[n][c] == top ? 1.0f : ex2(m[n][c] - top);
                        m[n][c] = top;
                        l[n][c] *= alpha;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            o[n][k][c] *= alpha;
                            o[n][k][2 + c] *= alpha;
                        }
                    }
            }
            uint32_t pb[NT][2], see01[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = ex2(sc[n][e] - (m[n][e & 1] == -INFINITY ? 0.0f : m[n][e & 1]));
                l[n][0] = __fmaf_rn(w[0] + w[2], ivs, l[n][0]);
                l[n][1] = __fmaf_rn(w[1] + w[3], ivs, l[n][1]);
                pb[n][0] = transpose8x8(pack_weights(w[0], w[1]));
                pb[n][1] = transpose8x8(pack_weights(w[2], w[3]));
            }
            uint32_t bad[4][DH / 32];
            bool any_bad = false;
            if (!full) {
                // NaN value codes in a slice that some row does not see wholly: a masked one must
                // not reach the sums (0 * NaN), a visible one must
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int w = 0; w < DH / 32; ++w) {
                        const uint32_t nb = e4m3_nan_bits(sl.v[r][w]) >> 7;
                        bad[r][w] = nb * 0x38u;  // 1.0 where NaN
                        sl.v[r][w] &= ~(nb * 0xffu);
                        any_bad |= nb != 0;
                    }
                any_bad = __any_sync(FULL_MASK, any_bad);
                if (any_bad) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        see01[n][0] = transpose8x8(pack16(sc[n][0] == -INFINITY ? 0.0f : 1.0f, sc[n][1] == -INFINITY ? 0.0f : 1.0f, true));
                        see01[n][1] = transpose8x8(pack16(sc[n][2] == -INFINITY ? 0.0f : 1.0f, sc[n][3] == -INFINITY ? 0.0f : 1.0f, true));
                    }
                }
            }
#pragma unroll
            for (int w = 0; w < DH / 32; ++w) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // channels (4w + 2h, 4w + 2h + 1) of the lane's run: rows g and g + 8 of M tile 2w + h
                    const uint32_t lo = __byte_perm(sl.v[0][w], sl.v[1][w], h ? 0x7362 : 0x5140);
                    const uint32_t up = __byte_perm(sl.v[2][w], sl.v[3][w], h ? 0x7362 : 0x5140);
                    const uint32_t a0 = e4m3x2_to_half2(lo & 0xffffu), a1 = e4m3x2_to_half2(lo >> 16);
                    const uint32_t a2 = e4m3x2_to_half2(up & 0xffffu), a3 = e4m3x2_to_half2(up >> 16);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16(o[n][2 * w + h], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                }
            }
            if (any_bad) {
#pragma unroll
                for (int w = 0; w < DH / 32; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t lo = __byte_perm(bad[0][w], bad[1][w], h ? 0x7362 : 0x5140);
                        const uint32_t up = __byte_perm(bad[2][w], bad[3][w], h ? 0x7362 : 0x5140);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma_f16(d, e4m3x2_to_half2(lo & 0xffffu), e4m3x2_to_half2(lo >> 16), e4m3x2_to_half2(up & 0xffffu),
                                    e4m3x2_to_half2(up >> 16), see01[n][0], see01[n][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (d[e] > 0.0f) o[n][2 * w + h][e] = __uint_as_float(0x7fc00000u);
                        }
                    }
            }
            __syncwarp();
        }

        // ---- join the warps ------------------------------------------------------------------
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float sum = l[n][c];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(FULL_MASK, sum, off);
                const int row = 8 * n + 2 * t + c;
                if (row < rows) {
                    if (g == 0) {
                        sm.m[warp][row] = m[n][c];
                        sm.l[warp][row] = sum;
                    }
#pragma unroll
                    for (int k = 0; k < KS; k += 2)
                        *reinterpret_cast<float4 *>(&sm.o[warp][row][g * (DH / 8) + 2 * k]) =
                            make_float4(o[n][k][c], o[n][k][2 + c], o[n][k + 1][c], o[n][k + 1][2 + c]);
                }
            }
        __syncthreads();
        const bool whole = j0 == 0 && j1 == span.count;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (first ? 0 : 1);
        for (int i = threadIdx.x; i < rows * (DH / 4); i += NW * 32) {
            const int row = i / (DH / 4), c = 4 * (i % (DH / 4));
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; ++w) top = fmaxf(top, sm.m[w][row]);
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = sm.m[w][row] == -INFINITY ? 0.0f : ex2(sm.m[w][row] - top);
                const float4 v = *reinterpret_cast<const float4 *>(&sm.o[w][row][c]);
                if (sm.m[w][row] == -INFINITY && sm.l[w][row] == 0.0f) continue;
                sum = __fmaf_rn(sm.l[w][row], f, sum);
                acc.x = __fmaf_rn(v.x, f, acc.x);
                acc.y = __fmaf_rn(v.y, f, acc.y);
                acc.z = __fmaf_rn(v.z, f, acc.z);
                acc.w = __fmaf_rn(v.w, f, acc.w);
            }
            if (whole) {
                const float o4[4] = {acc.x, acc.y, acc.z, acc.w};
                store_row<4>(p, s, qt * R + row, hk, c, DH, o4, top, sum);
            } else {
                *reinterpret_cast<float4 *>(part.o + (slot * R + row) * DH + c) = acc;
                if (c == 0) *reinterpret_cast<float2 *>(part.ml + (slot * R + row) * 2) = make_float2(top, sum);
            }
        }
        first = false;
        if (j1 < span.count) break;
        u0 += EXTRA + span.count;
        j0 = 0;
        if (u0 + EXTRA < hi) next_unit(p, s, R, b, qt, hk);
    }
    if (p.status) {
        flags = __reduce_or_sync(FULL_MASK, flags);
        if (flags && lane == 0) atomicOr(p.status, flags);
    }
}

// Joins the partial rows of the units that a boundary between two CTAs cuts: boundary i does it for the unit
// whose second part it opens.  G warps take a row (their lanes DH / 32 channels each, a warp every G-th part):
// 8 where few units of few rows have parts on many SMs, whose loads are then in flight together, 2 where many
// units have few, 1 for the many rows and few parts of the tensor-memory kernel.
template <int DH, int G>
__global__ void __launch_bounds__(256, 5) k_attention_kv8_join(const AttnKV8Params p, int ctas, int R)
{
    constexpr int CPL = DH / 32;
    __shared__ float s_sum[8], s_acc[8][DH];
    // the next grid waits for this one to end: blocks of it that came earlier took a fifth longer for it all
    wait_prior_grid();
    const KV8Partials part(p.workspace, ctas, R, DH);
    const int i = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const KV8Meta me = part.meta[i], prev = part.meta[i - 1];
    if (me.j0 == 0 || (prev.j0 > 0 && prev.u0 == me.u0)) return;
    const KV8Seq s = kv8_seq_checked(p.x, me.b);  // asked for before the parts are counted
    int count = 2;  // CTA i - 1, i, and those that go on with the unit
    for (bool on = true; on; ) {
        const int k = i - 1 + count + lane;
        const bool goes = k < ctas && part.meta[k].j0 != 0 && part.meta[k].u0 == me.u0;
        const int n = __ffs(~__ballot_sync(FULL_MASK, goes)) - 1;  // -1: all 32
        count += n < 0 ? 32 : n;
        on = n < 0;
    }
    const int rows = min(R, s.n * p.ratio - me.qt * R);
    const int64_t first = 2 * static_cast<int64_t>(i - 1) + (prev.u0 == me.u0 ? 0 : 1);
    auto slot = [&](int k) { return k == 0 ? first : 2 * static_cast<int64_t>(i - 1 + k); };
    for (int row0 = blockIdx.y * (8 / G); row0 < rows; row0 += gridDim.y * (8 / G)) {
        const int row = min(row0 + warp / G, rows - 1);  // warps without a row do the last one too, and do not store it
        float top = -INFINITY;
        for (int k = lane; k < count; k += 32) top = fmaxf(top, part.ml[(slot(k) * R + row) * 2]);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
        float acc[CPL] = {}, sum = 0.0f;
#pragma unroll 8
        for (int k = warp % G; k < count; k += G) {
            const float2 ml = *reinterpret_cast<const float2 *>(part.ml + (slot(k) * R + row) * 2);
            const float *src = part.o + (slot(k) * R + row) * DH + CPL * lane;
            float v[CPL];
            if (CPL == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(src);
                v[0] = x.x;
                v[1] = x.y;
                v[CPL - 2] = x.z;
                v[CPL - 1] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(src);
                v[0] = x.x;
                v[1] = x.y;
            }
            // a part that saw nothing has zeros
            const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - top);
            sum = __fmaf_rn(ml.y, f, sum);
#pragma unroll
            for (int c = 0; c < CPL; ++c) acc[c] = __fmaf_rn(v[c], f, acc[c]);
        }
        if (G > 1) {
            __syncthreads();  // the row before's have been read
            if (lane == 0) s_sum[warp] = sum;
#pragma unroll
            for (int c = 0; c < CPL; ++c) s_acc[warp][CPL * lane + c] = acc[c];
            __syncthreads();
            if (warp % G > 0 || row0 + warp / G >= rows) continue;
            const int n = min(G, count);
            for (int k = 1; k < n; ++k) {
                sum += s_sum[warp + k];
#pragma unroll
                for (int c = 0; c < CPL; ++c) acc[c] += s_acc[warp + k][CPL * lane + c];
            }
        }
        if (row0 + warp / G < rows) store_row<CPL>(p, s, me.qt * R + row, me.hk, CPL * lane, DH, acc, top, sum);
    }
}

template <int DH, int NT>
cudaError_t launch(const AttnKV8Params &p, const DeviceInfo &dev, cudaStream_t stream)
{
    constexpr int NW = 4, PER_SM = NT == 1 ? 3 : 2;
    constexpr int smem = NW * sizeof(Ring<DH>) + sizeof(MergeSmem<DH, NT, NW>);
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t a = allow_smem(allowed, k_attention_kv8<DH, NT, NW>, smem, dev.ordinal);
    if (a != cudaSuccess) return a;
    const int ctas = dev.num_sms * PER_SM < KV8_MAX_CTAS ? dev.num_sms * PER_SM : KV8_MAX_CTAS;
    const cudaError_t e = launch_after_prior(k_attention_kv8<DH, NT, NW>, dim3(ctas), dim3(NW * 32), smem, stream, p);
    if (e != cudaSuccess) return e;
    return attention_kv8_join_launch(p, DH, ctas, 8 * NT, stream);
}

}  // namespace

cudaError_t attention_kv8_join_launch(const AttnKV8Params &p, int d_h, int ctas, int R, cudaStream_t stream)
{
    const auto launch_join = [&](auto kern, int y) { return launch_after_prior(kern, dim3(ctas - 1, y), dim3(256), 0, stream, p, ctas, R); };
    if (R > 32) return d_h == 64 ? launch_join(k_attention_kv8_join<64, 1>, 16) : launch_join(k_attention_kv8_join<128, 1>, 16);
    if (static_cast<int64_t>(p.x.B) * p.Hkv * 8 <= ctas)
        return d_h == 64 ? launch_join(k_attention_kv8_join<64, 8>, R / 2) : launch_join(k_attention_kv8_join<128, 8>, R / 2);
    return d_h == 64 ? launch_join(k_attention_kv8_join<64, 2>, R / 8) : launch_join(k_attention_kv8_join<128, 2>, R / 8);
}

size_t attention_kv8_workspace(int64_t T, int B, int Hq, int Hkv, int d_h)
{
    if (T <= 0 || B <= 0) return 0;
    return kv8_takes_tc(T, B, Hq / Hkv) ? KV8Partials::bytes(KV8_TC_MAX_CTAS, KV8_TC_ROWS, d_h)
                                        : KV8Partials::bytes(KV8_MAX_CTAS, 24, d_h);
}

cudaError_t attention_kv8_launch(const AttnKV8Params &p, int d_h, const DeviceInfo &dev, cudaStream_t stream)
{
    if (kv8_takes_tc(p.x.T, p.x.B, p.ratio)) return attention_kv8_tc_launch(p, d_h, dev, stream);
    // Query rows of a unit: what a sequence has.  The host does not know the counts; where they cannot all be
    // alike it goes by 4/3 of their mean: 8 rows more in a unit take 1.3 times as long (16 x 8000 tokens: 59,
    // 74, 101 us), a second unit for the sequences that have more twice, so a third of them may.
    const bool alike = !p.x.cu || p.x.T % p.x.B == 0;
    const int64_t rows = alike ? p.x.T / p.x.B * p.ratio : 4 * p.x.T * p.ratio / (3 * static_cast<int64_t>(p.x.B));
    cudaError_t e;
    if (rows <= 8)
        e = d_h == 64 ? launch<64, 1>(p, dev, stream) : launch<128, 1>(p, dev, stream);
    else if (rows <= 16)
        e = d_h == 64 ? launch<64, 2>(p, dev, stream) : launch<128, 2>(p, dev, stream);
    else
        e = d_h == 64 ? launch<64, 3>(p, dev, stream) : launch<128, 3>(p, dev, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qkq
