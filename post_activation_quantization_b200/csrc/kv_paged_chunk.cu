// kv_paged_chunk.cu -- paged attention of many query rows to a K/V head: prompts, chunks of prompts.
//
// Two contractions on the fifth-generation tensor cores, S = q' K^T and O += W V, with the softmax between
// them in registers (one pass over the positions, running maximum and sum).  A CTA holds two tiles of 128
// query rows (a row is a token and a head of the K/V head's group) and walks the positions in tiles of
// 128; all 512 tensor-memory columns: S of both tiles (W replaces it in place, as fp16) and O of both.
//   warps 0-3, 4-7    softmax of tile 0 / 1: one thread to a row
//   warps 8-11        expand the packed codes of K and V into shared memory, as fp16
//   warp 12           issues the MMAs of both (warps 13-15 fill its warpgroup)
// The two tiles share K and V and take turns on the tensor core: one's softmax runs while the other's
// products do.  The codes come from global memory a tile ahead, are masked in place (kv_paged_attn.cuh) and
// brought to small exact fp16 numbers by one fused multiply-add per two: K's relative to the first positions' mean (a shift
// of all scores of a row, which the softmax does not see; S, and what the queries' rounding does to it, then have the size
// of the scores' spread), V's relative to the code nearest to the channel's zero point.
// Queries come from a first kernel as finished operand tiles, already scaled (q' = q s) and in the 128-byte swizzle.
// For outputs of 16 bits W is one fp16, and without sums q' is too: 2^-11 at most of each, either way, which takes
// an fp16 output's error from 2.1e-4, its own rounding, to 2.1e-4 to 2.7e-4; the rows' sums take the weights before that
// rounding, in fp32.
// Where the scores must be good to fp32 (fp32 queries, or running sums of weights), q' has two fp16 parts and S takes two
// products.  fp32 outputs have W in two parts as well, tiles of 64 positions, and the products of a tile are added to O by
// the softmax's threads: the tensor core's own additions are cut off at the accumulator's last bit, and the many of a long
// row would all err to the same side (4e-6 after 1287 positions, measured).
//
// Measured (calls one behind another, each on other inputs) at 3 chunks of about 2048 tokens over about 6000 positions, 32 heads
// of 128, 3 bits, fp16: 503 us (34 of them the queries' kernel), 820 TFLOP/s, 0.50 of the tensor core's measured peak.  No
// unit is full (tensor core 0.46, special functions 0.40, issue slots 0.44): a tile's W V begins when all its weights are
// there, and its next scores when W V is done, so that the two tiles in turn leave both idle about half of the time.
//
// Running sums: a third kernel goes over the positions again with the rows' maxima and sums known: tiles of 128
// positions are the row operand, S^T = K q'^T, so that a thread owns a position and adds its weights in registers,
// row tile by row tile, in a fixed order.
// 2 chunks of 1024 tokens over about 8100 positions, 32 heads over 8, 4 bits, bf16: 600 us (each kernel by itself: queries 19,
// attention 345 in 1.7 waves of CTAs, sums 258).
#include <algorithm>
#include <type_traits>

#include "kv_paged_attn.cuh"
#include "tc.cuh"

namespace rptq {

constexpr int CH_M = 128, CH_KEYS = 128;
constexpr int CH_SOFT_WARPS = 8, CH_PROD_WARPS = 4;
constexpr int CH_PROD0 = CH_SOFT_WARPS, CH_MMA0 = CH_PROD0 + CH_PROD_WARPS;
constexpr int CH_THREADS = 32 * (CH_MMA0 + 4);  // whole warpgroups: registers are moved between them
constexpr uint32_t CH_SLAB = CH_M * 128;  // 128 rows of 64 fp16
// Weights are held as 2^y, y = x - m + shift for a reference m that follows the running maximum (it moves when some y passes
// CH_YMAX); fp16's smallest step is then 2^-(24 + shift) of a weight at the reference, and a weight, however small, may be off
// by half of that.  Outputs of 16 bits take CH_PSHIFT, which lets the maximum grow by 2^10 before O is scaled again (2^-30 of the largest
// weight for each position: 2^-13 over 131072), and the largest score itself for m: its weight is a power of two and has no
// rounding.  fp32 outputs, whose weights have two parts and whose O is scaled at every tile in any case, take
// CH_PSHIFT32, and an integer for m: shift - m and the factors are exact.  Running sums beside outputs of 16 bits need both, so
// there y = x - m rounds once, and 2^y is multiplied by 2^CH_PSHIFT (exact).
constexpr int CH_PSHIFT = 5, CH_PSHIFT32 = 14;
constexpr float CH_YMAX = 15.f;

// 2^y of two exponents on the FMA pipe: y = n + f with n the nearest integer (the sum with 1.5 * 2^23 holds it in its
// low bits), 2^f on [-1/2, 1/2] by the cubic of least relative error (7.5e-5, fitted for this; a weight's fp16 rounding
// is up to 4.9e-4), n added to the exponent.  y below -126 counts as -126, a masked one too: its weight is not 0 but 2^-126.  The special-function unit gives 16 results a clock
// and SM, which the tensor core's two products of a tile take no longer than: one weight in CH_POLY comes from here.
__device__ __forceinline__ f32x2 exp2_poly(f32x2 y)
{
    y = mk2(fmaxf(lo2(y), -126.f), fmaxf(hi2(y), -126.f));
    const f32x2 t = add2(y, mk2(MAGIC_RINT, MAGIC_RINT));
    const f32x2 f = fma2(add2(t, mk2(-MAGIC_RINT, -MAGIC_RINT)), mk2(-1.f, -1.f), y);
    f32x2 p = fma2(f, mk2(0.05517167f, 0.05517167f), mk2(0.24261112f, 0.24261112f));
    p = fma2(p, f, mk2(0.69326099f, 0.69326099f));
    p = fma2(p, f, mk2(0.99992807f, 0.99992807f));
    return mk2(__uint_as_float(__float_as_uint(lo2(t)) * 0x800000u + __float_as_uint(lo2(p))),
               __uint_as_float(__float_as_uint(hi2(t)) * 0x800000u + __float_as_uint(hi2(p))));
}
constexpr int CH_POLY = 8;  // (measured at 2048 tokens, 32 heads: none 537 us, 1 in 8 517, 1 in 4 550, 1 in 2 589)

// What the chunk kernels read besides PagedAttnDev.
struct ChunkDev {
    PagedAttnDev a;
    const uint8_t *tiles;  // operand tiles of q': [H, slots, parts, D / 64, 128 rows, 128 bytes]
    float *cx;             // [H, slots, 128]: base-2 score of a row = cx * S
    int64_t slots;         // tile slots of a head
};

// Tile slots of a head: sequence b's tiles of `rows` rows start at slot start[b] * G / rows + b (each sequence ends
// in at most one partial tile).  The sequence of a slot; the caller checks what it gets.
__device__ __forceinline__ int64_t chunk_base(const Paged &p, int b, int G, int rows)
{
    return (int64_t)p.start[b] * G / rows + b;
}
__device__ __forceinline__ int chunk_sequence(const Paged &p, int64_t slot, int G, int rows)
{
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (chunk_base(p, m, G, rows) <= slot)
            lo = m;
        else
            hi = m;
    }
    return lo;
}

template <int BITS, int D>
struct ChunkQ {
    using KP = KPairs<BITS, D>;
    // column of channel d in the order of the expanded codes, and the bit position of its code
    __device__ static void column(int d, int &col, int &pos)
    {
        const int t = d / (D / 4), c = d % (D / 4);
        col = pos = 0;
#pragma unroll
        for (int i = 0; i < KP::N; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (KP::code(i, e) == c) col = t * (D / 4) + 2 * i + e, pos = KP::pos(i, e);
    }
};

// N consecutive elements (2 or 4, aligned to their size) of a tensor of run-time type, as they lie and as numbers
template <int N>
__device__ __forceinline__ void load_raw(const void *p, int dtype, int64_t at, uint32_t (&w)[N])
{
    if (dtype == RPTQ_F32) {
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const float *>(p) + at + k);
            w[k] = u.x, w[k + 1] = u.y;
        }
    } else if constexpr (N == 4) {
        const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + at);
        w[0] = u.x, w[1] = u.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + at);
    }
}
template <int N>
__device__ __forceinline__ void raw_floats(const uint32_t (&w)[N], int dtype, float (&v)[N])
{
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        if (dtype == RPTQ_F32) {
            v[2 * k] = __uint_as_float(w[2 * k]), v[2 * k + 1] = __uint_as_float(w[2 * k + 1]);
        } else if (dtype == RPTQ_F16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
            v[2 * k] = f.x, v[2 * k + 1] = f.y;
        } else {
            v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
}

// ---- the queries as operand tiles -----------------------------------------------------------------------
// One CTA per (tile slot, head), a warp to a row.  PARTS = 1: fp16 of q' scaled so that the row's largest is in
// [2^14, 2^15); 2: and what that rounding leaves, as fp16 too: 22 bits of every element, or 2^-31 of the row's largest.  (Two integers on one grid
// relative to the row's largest would keep the sums of the first part exact, but a row with an outlier then leaves its
// other channels few bits: 3.6e-6 of the running sums instead of 2e-8, measured.)
constexpr int CQ_THREADS = 256;
template <int BITS, int D, int PARTS>
__global__ void __launch_bounds__(CQ_THREADS)
    paged_chunk_queries(const ChunkDev c, uint8_t *__restrict__ tiles)
{
    constexpr int CPL = D / 32;
    constexpr uint32_t BYTES = PARTS * (D / 64) * CH_SLAB;
    extern __shared__ __align__(16) uint8_t tile[];
    __shared__ float s_s[D];
    __shared__ uint32_t s_at[D];  // byte of channel d in a row of the tile (before the swizzle)
    __shared__ float s_down[D];   // 2^-pos of its code
    const PagedAttnDev &a = c.a;
    const Paged &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t slot = blockIdx.x % c.slots;
    const int h = (int)(blockIdx.x / c.slots);
    const int b = chunk_sequence(p, slot, a.G, CH_M);
    int s0, n, L;
    if (!paged_sequence(p, b, s0, n, L)) return;
    const int64_t i = slot - chunk_base(p, b, a.G, CH_M);
    const int64_t rows = (int64_t)n * a.G - i * CH_M;
    if (i < 0 || rows <= 0) return;
    // Each warp's rows, U at a time, their loads together and a turn ahead.  (Loads of four rows at the turn's start: 52 us at
    // 6144 rows of 32 heads against 34.)
    constexpr int U = 4, W = CQ_THREADS / 32;
    uint32_t raw[U][CPL];
    auto fetch = [&](int r0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = (int)i * CH_M + r0 + u, tok = row / a.G, j = row - tok * a.G;
            const int64_t at = (int64_t)(s0 + tok) * a.q_stride + (int64_t)(h * a.G + j) * D + lane * CPL;
#pragma unroll
            for (int k = 0; k < CPL; ++k) raw[u][k] = 0;
            if (r0 + u < rows) load_raw<CPL>(a.q, a.dtype, at, raw[u]);
        }
    };
    fetch(warp * U);
    for (int d = tid; d < D; d += CQ_THREADS) {
        int col, pos;
        ChunkQ<BITS, D>::column(d, col, pos);
        s_s[d] = a.kt.sk[cluster_of(a.kt.ck, h * D + d, a.kt.g, p.err)];
        s_at[d] = (col >> 6) * CH_SLAB + (col & 63) * 2;
        s_down[d] = 1.f / (float)(1 << pos);
    }
    __syncthreads();
    float sc[CPL], down[CPL];  // of the lane's channels
    uint32_t to[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) sc[k] = s_s[lane * CPL + k], down[k] = s_down[lane * CPL + k], to[k] = s_at[lane * CPL + k];
    for (int r0 = warp * U; r0 < CH_M; r0 += W * U) {
        float v[U][CPL], m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            raw_floats<CPL>(raw[u], a.dtype, v[u]);
            m[u] = 0.f;
#pragma unroll
            for (int k = 0; k < CPL; ++k) {
                v[u][k] *= sc[k];
                m[u] = fmaxf(m[u], fabsf(v[u][k]));
            }
        }
        if (r0 + W * U < CH_M) fetch(r0 + W * U);
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u) m[u] = fmaxf(m[u], __shfl_xor_sync(FULL, m[u], o));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u;
            const int ex = max((int)(__float_as_uint(m[u]) >> 23) - 126, -100);  // m in [2^(ex - 1), 2^ex)
            const float up = __uint_as_float((uint32_t)(127 + 15 - ex) << 23);  // 2^(15 - ex): 15 - ex <= 115
            if (lane == 0) c.cx[((int64_t)h * c.slots + slot) * CH_M + r] = a.scale * LOG2E * __uint_as_float((uint32_t)(127 - 5 + ex) << 23);
#pragma unroll
            for (int k = 0; k < CPL; ++k) {
                const uint32_t sw = (to[k] + r * 128) ^ ((r & 7) << 4);  // piece c of a row sits at c ^ (row mod 8)
                const float f = v[u][k] * up * down[k];
                const __half hi = __float2half_rn(f);
                *reinterpret_cast<__half *>(tile + sw) = hi;
                if (PARTS == 2) *reinterpret_cast<__half *>(tile + (D / 64) * CH_SLAB + sw) = __float2half_rn(f - __half2float(hi));
            }
        }
    }
    __syncthreads();
    uint4 *dst = reinterpret_cast<uint4 *>(tiles + ((int64_t)h * c.slots + slot) * BYTES);
    for (uint32_t k = tid; k < BYTES / 16; k += CQ_THREADS) dst[k] = reinterpret_cast<const uint4 *>(tile)[k];
}

// ---- expansion of the codes -----------------------------------------------------------------------------
// A producer thread (0-127) has one quarter of every 32nd row of a tile of 64 or 128.  The eight lanes of one 16-byte store phase
// write eight different 16-byte columns of the swizzled tile: D = 128: two quarters (of one slab) of four rows;
// D = 64: four quarters of two rows.
template <int D>
__device__ __forceinline__ void chunk_share(int pt, int &r0, int &t)
{
    if (D == 128)
        t = (pt & 1) | ((pt >> 6) << 1), r0 = (pt >> 1) & 31;
    else
        t = pt & 3, r0 = pt >> 2;
}
// The pages of its N rows of the tile (of 32 N) at pos0, as the table has them; page 0 for one outside the pool.
template <int N>
__device__ __forceinline__ void chunk_pages(const Paged &p, int b, int pos0, int L, int r0, int (&ids)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int pos = pos0 + r0 + 32 * i;
        ids[i] = pos < L ? p.table[(int64_t)b * p.max_pages + (pos >> p.shift)] : 0;
    }
}
template <int N>
__device__ __forceinline__ void chunk_check(const Paged &p, int (&ids)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (ids[i] < 0 || ids[i] >= p.n_pages) {
            raise_error(p.err, RPTQ_DEVERR_PAGE);
            ids[i] = 0;
        }
}
// its rows' packed words ...
template <int BITS, int D, int N>
struct ChunkCodes {
    using KP = KPairs<BITS, D>;
    uint32_t w[N][KP::NW];
    // rows r0, r0 + 32, ... of the tile at pos0, in pages `ids`; zeros past the sequence
    __device__ __forceinline__ void read(const uint8_t *pages, const Paged &p, const int (&ids)[N], int H, int h, int pos0, int L,
                                         int r0, int t)
    {
        constexpr int RB = D * BITS / 8;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int pos = pos0 + r0 + 32 * i;
#pragma unroll
            for (int k = 0; k < KP::NW; ++k) w[i][k] = 0;
            if (pos < L) KP::read(pages + (paged_row(ids[i], H, h, p.shift) + (pos & ((1 << p.shift) - 1))) * RB, t, w[i]);
        }
    }
    // ... to shared memory: fp16 of D / 64 slabs of [32 N rows, 128 bytes] in the 128-byte swizzle
    template <typename F>
    __device__ __forceinline__ void write(uint32_t tile, int r0, int t, F shape) const
    {
        constexpr int PIECES = KP::N / 4;  // 16-byte pieces of a quarter
        const int slab = t * PIECES / 8, c0 = t * PIECES % 8;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t x[KP::N];
            KP::expand(w[i], x);
            shape(x);
            const int r = r0 + 32 * i;
            const uint32_t row = tile + slab * N * 4096 + r * 128;
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
                const uint32_t at = row + (((c0 + j) ^ (r & 7)) << 4);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[4 * j]), "r"(x[4 * j + 1]),
                             "r"(x[4 * j + 2]), "r"(x[4 * j + 3])
                             : "memory");
            }
        }
    }
};

// What is taken off K's codes of quarter t, negated: the mean of the first 16 positions' (of the last one's again where there
// are fewer; all of one page), any choice being a shift of all scores of a row.  In sixteenths: exact in fp16.
template <int BITS, int D>
__device__ __forceinline__ void chunk_reference(const PagedAttnDev &a, int b, int h, int t, int L, uint32_t (&ref)[KPairs<BITS, D>::N])
{
    constexpr int N = KPairs<BITS, D>::N, RB = D * BITS / 8;
    const Paged &p = a.p;
    const uint8_t *rows = a.kq + paged_row(max(paged_page(p, b, 0), 0), a.H, h, p.shift) * RB;
    constexpr int STEP = D == 128 ? 2 : 4;  // lanes of a quarter (chunk_share): every STEP-th; each reads STEP / 2 of the rows
    const int r = (threadIdx.x & 31) / STEP;
    uint32_t x[N];
    KPairs<BITS, D>::load(rows + min(r, L - 1) * RB, t, x);
#pragma unroll
    for (int i = 0; i < N; ++i) ref[i] = code_up(x[i]);
    if (STEP == 4) {
        KPairs<BITS, D>::load(rows + min(r + 8, L - 1) * RB, t, x);
#pragma unroll
        for (int i = 0; i < N; ++i) ref[i] = code_up_plus(x[i], ref[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __half2 v = *reinterpret_cast<const __half2 *>(&ref[i]);
#pragma unroll
        for (int o = STEP; o < 32; o <<= 1) v = __hadd2(v, __shfl_xor_sync(FULL, v, o));
        v = __hmul2(v, __float2half2_rn(-1.f / 16.f));
        ref[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
}

// ---- attention --------------------------------------------------------------------------------------------
template <int D, int QP, int PP>  // parts of q' and of W
struct ChunkShape {
    static constexpr int SLABS = D / 64;
    static constexpr int KEYS = PP == 2 ? 64 : 128;  // positions of a tile
    static constexpr uint32_t KV_SLAB = KEYS * 128, KV = SLABS * KV_SLAB;  // a K or V tile
    static constexpr uint32_t QT = QP * SLABS * CH_SLAB;                   // a query tile
    static constexpr int STAGES = QP == 2 && PP == 1 && D == 128 ? 1 : 2;  // what 227 KB leave (a second one of K alone: no faster)
    static constexpr uint32_t SMEM = 1024 + 2 * QT + 2 * STAGES * KV;
    static constexpr uint32_t O_COL = 256;  // O of tile g at O_COL + g * D
};

template <int BITS, int D, int QP, int PP>
__global__ void __launch_bounds__(CH_THREADS, 1)
    paged_chunk_kernel(const ChunkDev c)
{
    using S = ChunkShape<D, QP, PP>;
    using KP = KPairs<BITS, D>;
    constexpr int ST = S::STAGES, KEYS = S::KEYS;
    // the weights' shift: in their exponents, or by a product behind them (see CH_PSHIFT)
    constexpr bool AFTER = QP == 2 && PP == 1;
    constexpr int WSHIFT = PP == 2 ? CH_PSHIFT32 : CH_PSHIFT;
    constexpr float SHIFT = AFTER ? 0.f : (float)WSHIFT, YMAX = AFTER ? CH_YMAX - WSHIFT : CH_YMAX;
    constexpr int HALVES = D / 64;  // PP = 2: a tile's product, 64 channels at a time, lies beside S
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[4 * 2 + 4 * 2 + 2];
    __shared__ uint32_t tmem_slot;
    __shared__ float s_sv[D], s_zv[D];
    __shared__ int s_zc[D];
    const PagedAttnDev &a = c.a;
    const Paged &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // CTA: (block of 256 rows, head, part of the positions); the blocks of a sequence from its last one (the longest) on
    const int split = blockIdx.x % a.splits;
    const int64_t u = blockIdx.x / a.splits;
    const int h = (int)(u % a.H);
    const int64_t slot2 = u / a.H;
    const int b = chunk_sequence(p, slot2, a.G, 2 * CH_M);
    int s0, n, L;
    if (!paged_sequence(p, b, s0, n, L)) return;
    const int R = n * a.G, blocks = (R + 2 * CH_M - 1) / (2 * CH_M);
    const int64_t bi = slot2 - chunk_base(p, b, a.G, 2 * CH_M);
    if (bi < 0 || bi >= blocks) return;
    const int block = blocks - 1 - (int)bi;
    const int row0 = block * 2 * CH_M, rows = min(2 * CH_M, R - row0);
    const int nact = rows > CH_M ? 2 : 1;
    const int64_t qslot = (int64_t)h * c.slots + chunk_base(p, b, a.G, CH_M) + 2 * block;
    // tiles of positions: those that the last row sees, this part's share
    const int vis = max(0, L - n + (row0 + rows - 1) / a.G + 1);
    const int all = (vis + KEYS - 1) / KEYS;
    const int j0 = (int)((int64_t)all * split / a.splits), j1 = (int)((int64_t)all * (split + 1) / a.splits);

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sQ = base, sK = base + 2 * S::QT, sV = sK + ST * S::KV;
    const uint32_t bar = smem_u32(bars);
    const uint32_t k_full = bar, k_empty = bar + 16, v_full = bar + 32, v_empty = bar + 48;  // [2] each
    const uint32_t s_full = bar + 64, p_full = bar + 80, o_done = bar + 96, o_free = bar + 112, q_full = bar + 128, drain = bar + 136;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full + 8 * i, 32 * CH_PROD_WARPS);
            mbar_init(v_full + 8 * i, 32 * CH_PROD_WARPS);
            mbar_init(k_empty + 8 * i, 1);
            mbar_init(v_empty + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, CH_M);
            mbar_init(o_done + 8 * i, 1);
            mbar_init(o_free + 8 * i, CH_M);
        }
        mbar_init(q_full, 1);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    for (int d = tid; d < D; d += CH_THREADS) {
        const int k = cluster_of(a.kt.cv, h * D + d, a.kt.g, p.err);
        s_sv[d] = a.kt.sv[k];
        const int z = a.kt.zv[k], zc = zero_code(z, (1 << BITS) - 1);
        s_zv[d] = (float)(z - zc);
        s_zc[d] = zc;
    }
    if (warp == CH_MMA0) tc_alloc(smem_u32(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // 512 threads start with 128 registers each; a row of S takes 128: 2 * 168 + 112 + 64 = 4 * 128
    if (warp < CH_SOFT_WARPS) {
        reg_inc<168>();
        const int g = warp >> 2, quad = warp & 3;
        const int r = 32 * quad + lane, row = row0 + g * CH_M + r;  // the thread's row
        const bool live = g < nact && row < R;
        if (g < nact) {
            const uint32_t lanes = (uint32_t)(32 * quad) << 16;
            const uint32_t tS = tmem + lanes + (uint32_t)g * CH_M, tO = tmem + lanes + S::O_COL + (uint32_t)g * D;
            const float cx = c.cx[(qslot + g) * CH_M + r];
            const int vrow = live ? L - n + row / a.G + 1 : 0;                    // visible positions
            const int vmin = L - n + (row0 + g * CH_M + 32 * quad) / a.G + 1;     // of the warp's first row
            float m = -1e30f, off = live ? 1e30f : -INFINITY;
            f32x2 l2 = mk2(0.f, 0.f);
            bool ok = true;
            for (int j = j0; j < j1 && ok; ++j) {
                ok = __all_sync(FULL, mbar_wait_bounded(s_full + 8 * g, (j - j0) & 1, p.err));
                if (!ok) break;
                tc_fence_after();
                const int pos0 = j * KEYS;
                const bool whole = pos0 + KEYS <= vmin;
                float top = -INFINITY;
                uint32_t v[KEYS / 32][32];  // the row of S
#pragma unroll
                for (int q4 = 0; q4 < KEYS / 32; ++q4) tc_ld32_async(tS + 32 * q4, v[q4]);
                tc_wait_ld();
#pragma unroll
                for (int q4 = 0; q4 < KEYS / 32; ++q4) tc_loaded(v[q4]);
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < KEYS; ++k)
                        if (pos0 + k >= vrow) v[k / 32][k % 32] = 0xff800000u;  // -inf (cx > 0)
                }
#pragma unroll
                for (int k = 0; k < KEYS; k += 2)
                    top = max3f(top, __uint_as_float(v[k / 32][k % 32]), __uint_as_float(v[k / 32][k % 32 + 1]));
                // cx > 0, so the largest score is cx * the largest S
                const float ytop = fmaf(top, cx, off);
                float f = 1.f;
                if (__any_sync(FULL, ytop > YMAX)) {
                    if (live && ytop > SHIFT) {
                        const float mn = PP == 1 ? top * cx : ceilf(top * cx);
                        f = ex2(m - mn);
                        m = mn;
                        off = SHIFT - mn;
                        l2 = mul2(l2, mk2(f, f));
                    }
                    if (PP == 1 && j > j0) {  // O of the tiles so far (its products are complete: the scores waited for them)
#pragma unroll 1
                        for (int q8 = 0; q8 < D / 8; ++q8) {
                            uint32_t x[8];
                            tc_ld8(tO + 8 * q8, x);
#pragma unroll
                            for (int k = 0; k < 8; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
                            tc_st8(tO + 8 * q8, x);
                        }
                    }
                }
                const f32x2 cx2 = mk2(cx, cx), off2 = mk2(off, off);
#pragma unroll
                for (int q4 = 0; q4 < KEYS / 32; ++q4) {
                    uint32_t w[16], w2[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const f32x2 y = fma2(mk2(__uint_as_float(v[q4][2 * k]), __uint_as_float(v[q4][2 * k + 1])), cx2, off2);
                        // (precise weights stay with the finer function)
                        f32x2 e = QP == 1 && k % CH_POLY == CH_POLY - 1 ? exp2_poly(y) : mk2(ex2(lo2(y)), ex2(hi2(y)));
                        if (AFTER) e = mul2(e, mk2((float)(1 << WSHIFT), (float)(1 << WSHIFT)));
                        l2 = add2(l2, e);
                        w[k] = half2_bits(lo2(e), hi2(e));
                        if (PP == 2) {
                            const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                            w2[k] = half2_bits(lo2(e) - hf.x, hi2(e) - hf.y);
                        }
                    }
                    // W over 32 columns of S: 16 columns, its second part in the next 16
                    tc_st16(tS + 32 * q4, w);
                    if (PP == 2) tc_st16(tS + 32 * q4 + 16, w2);
                }
                tc_wait_st();
                tc_fence_before();
                lin_arrive(p_full + 8 * g);
                if constexpr (PP == 2) {  // O = f O + this tile's product
                    for (int hf = 0; hf < HALVES && ok; ++hf) {
                        ok = __all_sync(FULL, mbar_wait_bounded(o_done + 8 * g, ((j - j0) * HALVES + hf) & 1, p.err));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int q4 = 0; q4 < 2; ++q4) {
                            uint32_t x[32], o[32];
                            tc_ld32_async(tS + 64 + 32 * q4, x);
                            if (j > j0) tc_ld32_async(tO + 64 * hf + 32 * q4, o);
                            tc_wait_ld();
                            tc_loaded(x);
                            if (j > j0) {
                                tc_loaded(o);
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    x[k] = __float_as_uint(fmaf(__uint_as_float(o[k]), f, __uint_as_float(x[k])));
                            }
#pragma unroll
                            for (int k = 0; k < 2; ++k) tc_st16(tO + 64 * hf + 32 * q4 + 16 * k, reinterpret_cast<uint32_t(&)[16]>(x[16 * k]));
                        }
                        tc_wait_st();
                        tc_fence_before();
                        lin_arrive(o_free + 8 * g);
                    }
                }
            }
            // ---- the row's result ----
            if (PP == 1 && ok && j1 > j0) ok = mbar_wait_bounded(o_done + 8 * g, (j1 - j0 - 1) & 1, p.err);
            ok = __all_sync(FULL, ok);
            tc_fence_after();
            if (ok) {
                constexpr float UNSHIFT = 1.f / (float)(1 << WSHIFT);
                const float l = (lo2(l2) + hi2(l2)) * UNSHIFT;
                // The reference has moved: the row saw a position of this part.  (The sum does not tell: a masked weight from
                // exp2_poly is 2^-126, nothing beside a visible one but more than 0 without.)
                const bool sees = m > -1e30f || l != l;
                const int tok = row / a.G, jh = row - tok * a.G;
                const int64_t orow = (int64_t)(s0 + tok) * a.Hq + h * a.G + jh;
                const float inv = sees ? 1.f / l : 0.f;
#pragma unroll 1
                for (int q4 = 0; q4 < D / 32; ++q4) {
                    uint32_t v[32];
                    if (j1 > j0) {
                        tc_ld32(tO + 32 * q4, v);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = 0;
                    }
                    if (!live) continue;
                    float o[32];  // channels 32 q4 .. in order
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        constexpr int Q = D / 4;  // columns of a quarter
                        const int i = k % Q / 2, e = k & 1;
                        o[k / Q * Q + KP::code(i, e)] = __uint_as_float(v[k]) * ((float)(1 << (10 - KP::pos(i, e))) * UNSHIFT);
                    }
                    if (a.part != nullptr) {
                        float4 *dst = reinterpret_cast<float4 *>(a.part + ((int64_t)split * p.T * a.Hq + orow) * D + 32 * q4);
#pragma unroll
                        for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                        continue;
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = sees ? s_sv[32 * q4 + k] * (o[k] * inv - s_zv[32 * q4 + k]) : 0.f;
                    if (a.dtype == RPTQ_F32) {
                        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + orow * D + 32 * q4);
#pragma unroll
                        for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    } else {
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const __nv_bfloat162 bb = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
                            w[k] = a.dtype == RPTQ_F16 ? half2_bits(o[2 * k], o[2 * k + 1]) : *reinterpret_cast<const uint32_t *>(&bb);
                        }
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__half *>(a.out) + orow * D + 32 * q4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) dst[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    }
                }
                if (live && a.part != nullptr) {
                    float *ml = a.ml + ((int64_t)split * p.T * a.Hq + orow) * 2;
                    ml[0] = sees ? m : -INFINITY;
                    ml[1] = l;
                } else if (live && a.stat != nullptr) {
                    a.stat[2 * orow] = sees ? m : 0.f;
                    a.stat[2 * orow + 1] = inv;
                }
            }
        }
    } else if (warp < CH_MMA0) {
        // ---- producers ----
        reg_dec<112>();
        const int pt = tid - 32 * CH_PROD0;
        if (pt == 0) {
            const uint8_t *src = c.tiles + qslot * S::QT;
            mbar_expect_tx(q_full, nact * S::QT);
            for (uint32_t o = 0; o < nact * S::QT; o += CH_SLAB) bulk_g2s(sQ + o, src + o, CH_SLAB, q_full);
        }
        int r0, t;
        chunk_share<D>(pt, r0, t);
        bool ok = true;
        if (j1 > j0) {
            uint32_t ref[KP::N], zc[KP::N];  // what is taken off K's and V's codes
            chunk_reference<BITS, D>(a, b, h, t, L, ref);
#pragma unroll
            for (int i = 0; i < KP::N; ++i)
                zc[i] = half2_bits(code_offset(s_zc[t * (D / 4) + KP::code(i, 0)], KP::pos(i, 0)),
                                   code_offset(s_zc[t * (D / 4) + KP::code(i, 1)], KP::pos(i, 1)));
            ChunkCodes<BITS, D, KEYS / 32> kc, vc;
            int ids[KEYS / 32];  // pages of the tile whose codes are read next: themselves read a tile before that
            chunk_pages(p, b, j0 * KEYS, L, r0, ids);
            chunk_check(p, ids);
            kc.read(a.kq, p, ids, a.H, h, j0 * KEYS, L, r0, t);
            vc.read(a.vq, p, ids, a.H, h, j0 * KEYS, L, r0, t);
            chunk_pages(p, b, (j0 + 1) * KEYS, L, r0, ids);
            for (int j = j0; j < j1 && ok; ++j) {
                const int i = j - j0, st = i % ST;
                const uint32_t free_ph = ((uint32_t)(i / ST) & 1) ^ 1;
                if (!(ok = mbar_wait_bounded(k_empty + 8 * st, free_ph, p.err))) break;
                kc.write(sK + st * S::KV, r0, t, [&](uint32_t(&x)[KP::N]) {
#pragma unroll
                    for (int k = 0; k < KP::N; ++k) x[k] = code_up_plus(x[k], ref[k]);
                });
                fence_proxy_async_smem();
                lin_arrive(k_full + 8 * st);
                chunk_check(p, ids);
                if (j + 1 < j1) kc.read(a.kq, p, ids, a.H, h, (j + 1) * KEYS, L, r0, t);
                if (!(ok = mbar_wait_bounded(v_empty + 8 * st, free_ph, p.err))) break;
                vc.write(sV + st * S::KV, r0, t, [&](uint32_t(&x)[KP::N]) {
#pragma unroll
                    for (int k = 0; k < KP::N; ++k) x[k] = code_up_plus(x[k], zc[k]);
                });
                fence_proxy_async_smem();
                lin_arrive(v_full + 8 * st);
                if (j + 1 < j1) vc.read(a.vq, p, ids, a.H, h, (j + 1) * KEYS, L, r0, t);
                chunk_pages(p, b, (j + 2) * KEYS, L, r0, ids);
            }
        }
        if (pt == 0) mbar_wait_bounded(q_full, 0, p.err);  // no copy may be in flight when the CTA ends
    } else {
        // ---- MMA issue: the tiles in turn, each its W V of this turn and then its q' K^T of the next, so that one
        //      tile's products run during the other's softmax ----
        reg_dec<64>();
        if (warp == CH_MMA0 && lane == 0) {
            constexpr uint32_t qk = f16_idesc(CH_M, KEYS), pv = f16_idesc(CH_M, D) | IDESC_B_MN;
            const int count = j1 - j0;
            auto scores = [&](int g, int st) {
                const uint32_t q0 = sQ + g * S::QT;
#pragma unroll
                for (int part = 0; part < QP; ++part)
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc_mma_f16_ss(tmem + (uint32_t)g * CH_M,
                                      sw128_desc(q0 + (part * S::SLABS + kk / 4) * CH_SLAB) + 2 * (kk % 4),
                                      sw128_desc(sK + st * S::KV + kk / 4 * S::KV_SLAB) + 2 * (kk % 4), qk, (part | kk) != 0);
                tc_commit(s_full + 8 * g);
            };
            bool ok = mbar_wait_bounded(q_full, 0, p.err);
            if (ok && count > 0 && (ok = mbar_wait_bounded(k_full, 0, p.err))) {
                tc_fence_after();
                for (int g = 0; g < nact; ++g) scores(g, 0);
                tc_commit(k_empty);
            }
            for (int i = 0; i < count && ok; ++i) {
                const int st = i % ST, st1 = (i + 1) % ST;
                if constexpr (PP == 2) {  // each product where it is added from; then both tiles' next scores
                    constexpr uint32_t pv64 = f16_idesc(CH_M, 64) | IDESC_B_MN;
                    for (int hf = 0; hf < HALVES && ok; ++hf)
                        for (int g = 0; g < nact && ok; ++g) {
                            const uint32_t tS = tmem + (uint32_t)g * CH_M;
                            ok = hf == 0 ? mbar_wait_bounded(p_full + 8 * g, i & 1, p.err)
                                         : mbar_wait_bounded(o_free + 8 * g, (i * HALVES + hf - 1) & 1, p.err);
                            if (!ok) break;
                            if (hf == 0 && g == 0 && !(ok = mbar_wait_bounded(v_full + 8 * st, (uint32_t)(i / ST) & 1, p.err))) break;
                            tc_fence_after();
#pragma unroll
                            for (int part = 0; part < PP; ++part)
#pragma unroll
                                for (int kk = 0; kk < KEYS / 16; ++kk)
                                    tc_mma_f16_ts(tS + 64, tS + 32 * (kk >> 1) + 8 * (kk & 1) + 16 * part,
                                                  sw128_mn_desc(sV + st * S::KV + hf * S::KV_SLAB + kk * 2048, S::KV_SLAB), pv64, (part | kk) != 0);
                            tc_commit(o_done + 8 * g);
                            if (hf == HALVES - 1 && g == nact - 1) tc_commit(v_empty + 8 * st);
                        }
                    if (!ok || i + 1 == count) continue;
                    if (!(ok = mbar_wait_bounded(k_full + 8 * st1, (uint32_t)((i + 1) / ST) & 1, p.err))) break;
                    for (int g = 0; g < nact && ok; ++g) {
                        if (!(ok = mbar_wait_bounded(o_free + 8 * g, (i * HALVES + HALVES - 1) & 1, p.err))) break;
                        tc_fence_after();
                        scores(g, st1);
                        if (g == nact - 1) tc_commit(k_empty + 8 * st1);
                    }
                } else {
                    for (int g = 0; g < nact && ok; ++g) {
                        const uint32_t tS = tmem + (uint32_t)g * CH_M, tO = tmem + S::O_COL + (uint32_t)g * D;
                        if (!(ok = mbar_wait_bounded(p_full + 8 * g, i & 1, p.err))) break;
                        if (g == 0 && !(ok = mbar_wait_bounded(v_full + 8 * st, (uint32_t)(i / ST) & 1, p.err))) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < KEYS / 16; ++kk)
                            tc_mma_f16_ts(tO, tS + 32 * (kk >> 1) + 8 * (kk & 1),
                                          sw128_mn_desc(sV + st * S::KV + kk * 2048, S::KV_SLAB), pv, i > 0 || kk != 0);
                        tc_commit(o_done + 8 * g);
                        if (g == nact - 1) tc_commit(v_empty + 8 * st);
                        if (i + 1 == count) continue;
                        if (g == 0 && !(ok = mbar_wait_bounded(k_full + 8 * st1, (uint32_t)((i + 1) / ST) & 1, p.err))) break;
                        // S (and W in its place) is free once the products that read it are complete
                        if (!(ok = mbar_wait_bounded(o_done + 8 * g, i & 1, p.err))) break;
                        tc_fence_after();
                        scores(g, st1);
                        if (g == nact - 1) tc_commit(k_empty + 8 * st1);
                    }
                }
            }
            tc_commit(drain);  // tensor memory is released below: every issued product first
            mbar_wait_bounded(drain, 0, p.err);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == CH_MMA0) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

// ---- running sums -------------------------------------------------------------------------------------------
// One CTA per (sequence, head, 256 positions), all 512 tensor-memory columns: S^T of two tiles of 128 positions and a row
// tile, twice.  Warps 0-3 and 4-7 take the row tiles in turn; a thread
// has one position of each tile, so that what it reads of a row from shared memory (8 bytes for every lane: two clocks of the
// 128 bytes a clock) serves two weights.  Warp 8 issues the
// MMAs, warp 9 the copies of the query tiles (two in flight).
constexpr int CW_THREADS = 320, CW_TILES = 2;
template <int D>
struct WeightShape {
    static constexpr uint32_t QT = 2 * (D / 64) * CH_SLAB, KT = (D / 64) * CH_SLAB;
    static constexpr uint32_t SMEM = 1024 + 2 * QT + CW_TILES * KT;
};
template <int BITS, int D>
__global__ void __launch_bounds__(CW_THREADS, 1)
    paged_chunk_weights(const ChunkDev c, int blocks)
{
    using S = WeightShape<D>;
    using KP = KPairs<BITS, D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[9];
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) float2 s_row[2][2][CH_M];  // [group][turn][row]: cx, -(maximum + log2 of the sum)
    __shared__ int s_vis[2][2][CH_M];                   // visible positions
    __shared__ float2 s_sum[CH_M];
    const PagedAttnDev &a = c.a;
    const Paged &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blk = blockIdx.x % blocks, bh = blockIdx.x / blocks, b = bh / a.H, h = bh % a.H;
    int s0, n, L;
    if (!paged_sequence(p, b, s0, n, L)) return;
    const int R = n * a.G, first = blk * CW_TILES * CH_KEYS;
    if (R == 0 || first >= L) return;
    const int nact = first + CH_KEYS < L ? 2 : 1;  // tiles of positions
    const int64_t qslot = (int64_t)h * c.slots + chunk_base(p, b, a.G, CH_M);
    const int i0 = (int)((int64_t)max(0, first - (L - n)) * a.G / CH_M), i1 = (R + CH_M - 1) / CH_M;  // row tiles that see the block

    const uint32_t sQ = (smem_u32(smem_raw) + 1023u) & ~1023u, sK = sQ + 2 * S::QT;
    const uint32_t bar = smem_u32(bars);
    const uint32_t q_full = bar, q_empty = bar + 16, s_full = bar + 32, s_free = bar + 48, drain = bar + 64;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 1);
            mbar_init(q_empty + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(s_free + 8 * i, CH_M);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 8) tc_alloc(smem_u32(&tmem_slot), 512);
    const int g = warp >> 2;
    if (g < nact) {  // warps 0-3 and 4-7 expand a tile of positions each
        const int pos0 = first + g * CH_KEYS;
        int r0, t, ids[4];
        chunk_share<D>(tid & (CH_M - 1), r0, t);
        uint32_t ref[KP::N];
        chunk_reference<BITS, D>(a, b, h, t, L, ref);
        ChunkCodes<BITS, D, CH_KEYS / 32> kc;
        chunk_pages(p, b, pos0, L, r0, ids);
        chunk_check(p, ids);
        kc.read(a.kq, p, ids, a.H, h, pos0, L, r0, t);
        kc.write(sK + g * S::KT, r0, t, [&](uint32_t(&x)[KP::N]) {
#pragma unroll
            for (int k = 0; k < KP::N; ++k) x[k] = code_up_plus(x[k], ref[k]);
        });
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp < 8) {
        const int quad = warp & 3, r = 32 * quad + lane;
        const uint32_t tS = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)g * CW_TILES * CH_M;
        const int pos = first + r;  // and pos + 128
        // the thread's row of tile i
        auto info = [&](int i, float2 &f, int &vis) {
            const int row = i * CH_M + r;
            f = make_float2(0.f, -INFINITY);
            vis = 0;
            if (i >= i1 || row >= R) return;
            const int tok = row / a.G, j = row - tok * a.G;
            const float2 st = *reinterpret_cast<const float2 *>(a.stat + 2 * ((int64_t)(s0 + tok) * a.Hq + h * a.G + j));
            // scores are relative to those of K's mean, so the maximum is small enough for the sum's log to be added to it
            f = make_float2(c.cx[(qslot + i) * CH_M + r], st.y > 0.f ? log2f(st.y) - st.x : st.y == 0.f ? -INFINITY : st.y);
            vis = L - n + tok + 1;
        };
        f32x2 w = mk2(0.f, 0.f);  // of pos, pos + 128
        bool ok = true;
        float2 f;
        int vis;
        info(i0 + g, f, vis);
        for (int i = i0 + g, k = 0; i < i1; i += 2, ++k) {  // every warp takes every turn: the barrier counts them
            s_row[g][k & 1][r] = f;
            s_vis[g][k & 1][r] = vis;
            asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory");
            info(i + 2, f, vis);  // in flight during this turn
            ok = ok && __all_sync(FULL, mbar_wait_bounded(s_full + 8 * g, k & 1, p.err));
            if (!ok) continue;
            tc_fence_after();
            const bool whole = first + CW_TILES * CH_KEYS <= L - n + i * CH_M / a.G + 1;  // every row sees every position
            const float2 *rows = s_row[g][k & 1];
            const int *seen = s_vis[g][k & 1];
            auto add = [&](auto all) {
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    uint32_t u[32], v[32];
                    tc_ld32_async(tS + 32 * q4, u);
                    tc_ld32_async(tS + CH_M + 32 * q4, v);  // (of no use, and not used, without a second tile)
                    tc_wait_ld();
                    tc_loaded(u);
                    tc_loaded(v);
                    f32x2 t = mk2(0.f, 0.f);  // (32 at a time: the sum of 5384 rows in one chain was off by 1.6e-6)
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        const float2 s = rows[32 * q4 + q];
                        const f32x2 y = fma2(mk2(__uint_as_float(u[q]), __uint_as_float(v[q])), mk2(s.x, s.x), mk2(s.y, s.y));
                        f32x2 e = mk2(ex2(lo2(y)), ex2(hi2(y)));
                        if (!decltype(all)::value) {
                            const int vq = seen[32 * q4 + q];
                            e = mk2(pos < vq ? lo2(e) : 0.f, pos + CH_KEYS < vq ? hi2(e) : 0.f);
                        }
                        t = add2(t, e);
                    }
                    w = add2(w, t);
                }
            };
            if (whole)
                add(std::true_type());
            else
                add(std::false_type());
            tc_fence_before();
            lin_arrive(s_free + 8 * g);
        }
        if (g == 1) s_sum[r] = w;
        asm volatile("bar.sync 3, 256;" ::: "memory");
        if (g == 0) {
            const float2 o = s_sum[r];
            for (int t = 0; t < nact; ++t) {
                const int at = pos + t * CH_KEYS;
                if (at >= L) break;
                const int page = paged_page(p, b, at >> p.shift);
                if (page >= 0)
                    a.weights[paged_row(page, a.H, h, p.shift) + (at & ((1 << p.shift) - 1))] += t ? hi2(w) + o.y : lo2(w) + o.x;
            }
        }
    } else if (warp == 8) {
        if (lane == 0) {
            constexpr uint32_t id = f16_idesc(CH_M, CH_M);
            for (int i = i0, k = 0; i < i1; ++i, ++k) {
                const int st = k & 1;  // of the query tiles, and the group whose turn it is
                if (!mbar_wait_bounded(q_full + 8 * st, (k >> 1) & 1, p.err)) break;
                if (!mbar_wait_bounded(s_free + 8 * st, ((k >> 1) & 1) ^ 1, p.err)) break;
                tc_fence_after();
                for (int t = 0; t < nact; ++t)
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc_mma_f16_ss(tmem + (2 * st + t) * CH_M, sw128_desc(sK + t * S::KT + kk / 4 * CH_SLAB) + 2 * (kk % 4),
                                          sw128_desc(sQ + st * S::QT + (part * (D / 64) + kk / 4) * CH_SLAB) + 2 * (kk % 4), id,
                                          (part | kk) != 0);
                tc_commit(q_empty + 8 * st);
                tc_commit(s_full + 8 * st);
            }
            tc_commit(drain);
            mbar_wait_bounded(drain, 0, p.err);
        }
        __syncwarp();
    } else if (warp == 9) {
        if (lane == 0) {
            int issued = 0;
            for (int i = i0, k = 0; i < i1; ++i, ++k) {
                const int st = k & 1;
                if (!mbar_wait_bounded(q_empty + 8 * st, ((k >> 1) & 1) ^ 1, p.err)) break;
                const uint8_t *src = c.tiles + (qslot + i) * S::QT;
                mbar_expect_tx(q_full + 8 * st, S::QT);
                for (uint32_t o = 0; o < S::QT; o += CH_SLAB) bulk_g2s(sQ + st * S::QT + o, src + o, CH_SLAB, q_full + 8 * st);
                issued = k + 1;
            }
            for (int k = max(0, issued - 2); k < issued; ++k)  // no copy may be in flight when the CTA ends
                mbar_wait_bounded(q_full + 8 * (k & 1), (k >> 1) & 1, p.err);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

// ---- launch ---------------------------------------------------------------------------------------------------
namespace {
struct ChunkPlan {
    int qp, splits;
    int64_t slots, slots2;
    size_t tiles, cx, stat, part, total;  // offsets into the workspace, its size
};
ChunkPlan chunk_plan(int64_t T, int Hq, int H, int D, int dtype, int B, int max_len, int weights, int num_sms)
{
    ChunkPlan pl;
    const int64_t G = Hq / H, R = T * Hq;
    pl.qp = weights || dtype == RPTQ_F32 ? 2 : 1;
    pl.slots = T * G / CH_M + B;
    pl.slots2 = T * G / (2 * CH_M) + B;
    // the positions are split where the blocks of 256 rows leave SMs without one, each part at least four tiles
    const int64_t units = std::max<int64_t>(1, T * G / (2 * CH_M)) * H;
    pl.splits = (int)std::max<int64_t>(1, std::min<int64_t>({num_sms / units, max_len / (4 * CH_KEYS), 16}));
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    pl.tiles = 0;
    pl.cx = up((size_t)H * pl.slots * pl.qp * (D / 64) * CH_SLAB);
    pl.stat = pl.cx + up((size_t)H * pl.slots * CH_M * 4);
    pl.part = pl.stat + (weights ? up((size_t)R * 8) : 0);
    pl.total = pl.part + (pl.splits > 1 ? (size_t)pl.splits * R * (D + 2) * 4 : 0);
    return pl;
}

template <int BITS, int D, int QP, int PP>
cudaError_t launch_chunk(const ChunkDev &c, const ChunkPlan &pl, uint8_t *tiles, int B, cudaStream_t stream)
{
    constexpr size_t qsmem = (size_t)QP * (D / 64) * CH_SLAB;
    cudaError_t e = kernel_smem((const void *)paged_chunk_queries<BITS, D, QP>, qsmem);
    if (e == cudaSuccess) e = kernel_smem((const void *)paged_chunk_kernel<BITS, D, QP, PP>, ChunkShape<D, QP, PP>::SMEM);
    if (e != cudaSuccess) return e;
    paged_chunk_queries<BITS, D, QP><<<(unsigned)(pl.slots * c.a.H), CQ_THREADS, qsmem, stream>>>(c, tiles);
    paged_chunk_kernel<BITS, D, QP, PP>
        <<<(unsigned)(pl.slots2 * c.a.H * pl.splits), CH_THREADS, ChunkShape<D, QP, PP>::SMEM, stream>>>(c);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (pl.splits > 1 && (e = launch_paged_combine(c.a, D, stream)) != cudaSuccess) return e;
    if (c.a.weights != nullptr) {
        if constexpr (QP == 2) {
            if ((e = kernel_smem((const void *)paged_chunk_weights<BITS, D>, WeightShape<D>::SMEM)) != cudaSuccess) return e;
            const int blocks = (c.a.p.max_len + CW_TILES * CH_KEYS - 1) / (CW_TILES * CH_KEYS);
            paged_chunk_weights<BITS, D>
                <<<(unsigned)((int64_t)B * c.a.H * blocks), CW_THREADS, WeightShape<D>::SMEM, stream>>>(c, blocks);
        }
    }
    return cudaGetLastError();
}
template <int BITS, int D>
cudaError_t launch_chunk_prec(const ChunkDev &c, const ChunkPlan &pl, uint8_t *tiles, int B, cudaStream_t stream)
{
    if (c.a.dtype == RPTQ_F32) return launch_chunk<BITS, D, 2, 2>(c, pl, tiles, B, stream);
    if (pl.qp == 2) return launch_chunk<BITS, D, 2, 1>(c, pl, tiles, B, stream);
    return launch_chunk<BITS, D, 1, 1>(c, pl, tiles, B, stream);
}
}  // namespace

size_t paged_chunk_workspace(int64_t T, int Hq, int H, int D, int dtype, int B, int max_len, int weights, int num_sms)
{
    return chunk_plan(T, Hq, H, D, dtype, B, max_len, weights, num_sms).total;
}

cudaError_t launch_paged_chunk(const PagedAttnArgs &a)
{
    const ChunkPlan pl = chunk_plan(a.T, a.Hq, a.H, a.D, a.dtype, a.B, a.max_len, a.weights != nullptr, a.num_sms);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    ChunkDev c{};
    PagedAttnDev &d = c.a;
    d.p = Paged{a.start, a.lens, a.table, a.B, a.max_pages, a.shift, a.n_pages, a.T, a.max_q, a.max_len, a.err};
    d.q = a.q, d.out = a.out, d.dtype = a.dtype, d.Hq = a.Hq, d.H = a.H, d.G = a.Hq / a.H, d.q_stride = a.q_stride;
    d.kq = a.kq, d.vq = a.vq, d.kt = a.kt, d.scale = a.scale, d.weights = a.weights, d.splits = pl.splits;
    d.centred = (1 << a.bits) - 1;
    if (a.weights) d.stat = reinterpret_cast<float *>(ws + pl.stat);
    if (pl.splits > 1) {
        d.part = reinterpret_cast<float *>(ws + pl.part);
        d.ml = d.part + (int64_t)pl.splits * a.T * a.Hq * a.D;
    }
    uint8_t *tiles = ws + pl.tiles;
    c.tiles = tiles;
    c.cx = reinterpret_cast<float *>(ws + pl.cx);
    c.slots = pl.slots;
    if (a.bits == 4)
        return a.D == 128 ? launch_chunk_prec<4, 128>(c, pl, tiles, a.B, a.stream)
                          : launch_chunk_prec<4, 64>(c, pl, tiles, a.B, a.stream);
    return a.D == 128 ? launch_chunk_prec<3, 128>(c, pl, tiles, a.B, a.stream)
                      : launch_chunk_prec<3, 64>(c, pl, tiles, a.B, a.stream);
}

}  // namespace rptq
