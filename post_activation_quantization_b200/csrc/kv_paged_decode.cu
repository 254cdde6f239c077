// kv_paged_decode.cu -- paged attention of few query rows to a K/V head: decode steps, short chunks.
//
// Few rows make the packed codes the traffic (62 codes per clock and SM at 3 bits and 6.5 TB/s), and on
// the FMA pipe a code costs more instructions than that rate leaves.  Here the codes are the A operand of
// mma.sync.m16n8k16 (fp16, fp32 sums), taken from the packed bytes with one mask per two codes
// (kv_paged_attn.cuh), and the query rows are its 8 columns:
//     S [16 positions, 8 rows] = codes of K [16, D] x q'^T,       O [16 channels, 8 rows] = codes of V^T x w^T.
// The order of the channels inside a K step, and of the positions inside a block of 16, is free, so both
// operands are read from shared memory as they lie there.  Where the result must be good to fp16 or
// fp32, the 8 columns are fewer rows in two or three fp16 parts each.
//
// A CTA is four warps; warp w of part s of a (sequence, K/V head) takes the tiles of 32 positions
// s * 4 + w, + 4 * splits, ...  Each warp streams its tiles' K and V rows (contiguous in a page) with
// bulk copies into a ring of its own, keeps its own running maximum and sum, and needs no other warp until
// the end.  Up to eight parts of a (sequence, K/V head) are a cluster: its CTAs join their warps through distributed shared
// memory, write the outputs, and add to the running sums, each for the positions whose scores it kept.  More parts (long
// contexts, few heads) are joined by a second kernel.
//
// Measured (calls one behind another, each on other inputs): 16 sequences of 2048 positions, 32 heads of 128, 3 bits, fp16: 43 us,
// 2.4 TB/s of codes; 8 of about 2047, 96 heads, with sums: 61.5 us; 2 of about 131000, 32 heads over 8, 4 bits: 67.6 us,
// 3.85 TB/s.  No unit is full (first case: issue slots 0.52, ALU 0.52, matrix pipe 0.22, HBM 0.36 of 6.6 TB/s): a warp works a
// tile as one chain of dependent steps, and the 12 to 16 warps of an SM do not cover its latency.
#include <cooperative_groups.h>

#include <algorithm>

#include "kv_paged_attn.cuh"

namespace cg = cooperative_groups;

namespace rptq {

constexpr int DEC_WARPS = 4, DEC_THREADS = 32 * DEC_WARPS;
constexpr int DEC_TILE = 32;    // positions of a warp's tile: two blocks of 16
constexpr int DEC_STAGES = 3;   // tiles of a warp's ring: two on the way while one is worked (four: fewer CTAs to an SM, slower)
constexpr int DEC_CTAS_SM = 4;  // CTAs that share an SM: 128 registers a thread, 36 or 48 KB of rings
// Weights are held as 2^y, y = x - m + shift for a reference m that follows the running maximum (an integer not below it when
// it moves, which is when some y passes YMAX): 2^YMAX fits fp16, and its smallest step is 2^-(24 + shift) of a weight at the
// reference.  Outputs of 16 bits leave the maximum room to grow before the sums are scaled again (however small, a weight
// may be off by 2^-29 of the largest: 2^-12 over 131072 positions); fp32 ones give up room for bits: 2^-36, 2^-19 over 131072.  (8 sequences
// of 8000 positions, 32 heads over 8 of 128 / 64 over 8 of 64: shift 5 42.2 / 47.6 us, 10 42.4 / 48.2, 12 43.0 / 50.5, 14 45.4 / 57.8.)
constexpr int DEC_PSHIFT = 5, DEC_PSHIFT32 = 12;
constexpr float DEC_YMAX = 15.f, DEC_YMAX32 = 15.9f;

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of 16-bit elements across the warp
__device__ __forceinline__ uint32_t mat_trans(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// ---- V: one thread's D / 8 consecutive codes of two rows, code by code -----------------------------------
// x[i] holds code i of row a in the low half and of row b in the high half, both at bit pos(i).
template <int BITS, int D>
struct VCodes {
    static constexpr int N = D / 8, NW = (N * BITS + 31) / 32;
    __host__ __device__ static constexpr int pos(int i)
    {
        if (BITS == 4) return 4 * (i & 1);
        constexpr int P[16] = {0, 3, 6, 1, 4, 7, 2, 5, 8, 3, 6, 1, 4, 7, 2, 5};
        return P[i];
    }
    // the lane's codes of the row at `a`, from bit 0 of w[0]
    __device__ __forceinline__ static void load(const uint8_t *a, int g, uint32_t (&w)[NW])
    {
        if constexpr (BITS == 4 && D == 128) {
            const uint2 v = *reinterpret_cast<const uint2 *>(a + 8 * g);
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (BITS == 4) {
            w[0] = lds32(a + 4 * g);
        } else if constexpr (D == 128) {
            const uint8_t *p = a + ((6 * g) & ~3);
            const uint32_t s = 16 * (g & 1);
            const uint32_t wa = lds32(p), wb = lds32(p + 4);
            w[0] = __funnelshift_r(wa, wb, s);
            w[1] = wb >> s;
        } else {
            const int o = 3 * g;  // 24 bits at byte 3g
            const uint32_t wa = lds32(a + (o & ~3)), wb = lds32(a + ((o + 2) & ~3));
            w[0] = __funnelshift_r(wa, wb, 8 * (o & 3));
        }
    }
    __device__ __forceinline__ static void join(const uint32_t (&a)[NW], const uint32_t (&b)[NW], uint32_t (&x)[N])
    {
        if constexpr (BITS == 4) {
#pragma unroll
            for (int j = 0; j < N / 4; ++j) {
                const uint32_t m = prmt(a[j / 2], b[j / 2], (j & 1) ? 0x7632u : 0x5410u), u = m >> 8;
                x[4 * j] = m & 0x000F000Fu;
                x[4 * j + 1] = m & 0x00F000F0u;
                x[4 * j + 2] = u & 0x000F000Fu;
                x[4 * j + 3] = u & 0x00F000F0u;
            }
        } else {
            const uint32_t b0 = prmt(a[0], b[0], 0x5410u), b1 = prmt(a[0], b[0], 0x6521u), b2 = prmt(a[0], b[0], 0x7632u);
            x[0] = b0 & 0x00070007u;  // bits 0-15: codes 0, 1, 2
            x[1] = b0 & 0x00380038u;
            x[2] = b0 & 0x01C001C0u;
            x[3] = b1 & 0x000E000Eu;  // bits 8-23: codes 3, 4, 5
            x[4] = b1 & 0x00700070u;
            x[5] = b1 & 0x03800380u;
            x[6] = b2 & 0x001C001Cu;  // bits 16-31: codes 6, 7, 8
            x[7] = b2 & 0x00E000E0u;
            if constexpr (D == 128) {
                x[8] = b2 & 0x07000700u;
                const uint32_t b3 = prmt(__funnelshift_r(a[0], a[1], 24), __funnelshift_r(b[0], b[1], 24), 0x5410u);
                x[9] = b3 & 0x00380038u;  // bits 24-39: codes 9, 10
                x[10] = b3 & 0x01C001C0u;
                const uint32_t b4 = prmt(a[1], b[1], 0x5410u), b5 = prmt(a[1], b[1], 0x6521u);
                x[11] = b4 & 0x000E000Eu;  // bits 32-47: codes 11, 12, 13
                x[12] = b4 & 0x00700070u;
                x[13] = b4 & 0x03800380u;
                x[14] = b5 & 0x001C001Cu;  // bits 40-55: codes 14, 15
                x[15] = b5 & 0x00E000E0u;
            }
        }
    }
};

// RT rows to a column tile of 8.  PREC says what the result must be good to:
//   0 (bf16): q' and the weights one fp16, the codes as they are.  A product with a subnormal keeps 10 bits less in the tensor
//     core's sum (6e-5 of it), which is nothing in bf16.
//   1 (fp16, or running sums kept): q' in parts of 11 bits on one fixed grid -- with the codes multiplied up to
//     normal fp16 numbers every product and every sum of a part is exact -- so that a score has fp32's rounding and no
//     other; the weights in two fp16 parts, in columns that are there anyway (one: up to 4.1e-4 of an fp16 output, against
//     1.5e-4 to 3.1e-4, most of it the output's own rounding).  V's codes stay subnormals (6e-5).
//   2 (fp32): the same, V's codes multiplied up too, less the code nearest to the zero point.
// The grid's unit hangs on the row's largest |q'|: two parts, 22 bits of that, do for fp16 outputs; fp32 ones and the
// sums have three (a few large channels cost the others too much: 2e-5 of the output measured with two, 3e-7 with three).
// Columns: RT = 1: row 0's part t in column 2t, the odd ones empty (a lane then has half the softmax to do);
// RT = 2, 4: part * RT + row; RT = 8 (one part): the rows.
template <int BITS, int D, int RT, int NT, int PREC>
struct DecShape {
    static constexpr int ROWS = NT * RT;
    static constexpr int E = RT == 1 ? 1 : 2;  // columns of a lane that hold rows
    static constexpr int RB = D * BITS / 8;    // bytes of a packed row
    static constexpr uint32_t TILE = DEC_TILE * RB, STAGE = 2 * TILE;
    static constexpr size_t RING = (size_t)DEC_WARPS * DEC_STAGES * STAGE;
    static constexpr size_t JOIN = (size_t)DEC_WARPS * ROWS * (D + 2) * 4;  // the warps' results, when they are joined
    static constexpr size_t SMEM = RING > JOIN ? RING : JOIN;
    static constexpr int PARTS = PREC == 0 ? 1 : RT <= 2 ? 3 : 2;  // of q'
    // row in the tile, and part, of column `col`
    __device__ __forceinline__ static int row(int col) { return RT == 1 ? 0 : col & (RT - 1); }
    __device__ __forceinline__ static int part(int col) { return RT <= 2 ? col >> 1 : RT == 4 ? col >> 2 : 0; }
    __device__ __forceinline__ static bool used(int col) { return part(col) < PARTS && (RT != 1 || (col & 1) == 0); }
};

template <int BITS, int D, int RT, int NT, int PREC>
__global__ void __launch_bounds__(DEC_THREADS, NT == 1 ? (PREC == 2 ? 3 : DEC_CTAS_SM) : NT == 2 && PREC < 2 ? 3 : 2)
    paged_decode_kernel(const PagedAttnDev a)
{
    using S = DecShape<BITS, D, RT, NT, PREC>;
    using KP = KPairs<BITS, D>;
    using VC = VCodes<BITS, D>;
    constexpr int E = S::E;
    constexpr int PSHIFT = PREC == 2 ? DEC_PSHIFT32 : DEC_PSHIFT;
    constexpr float YMAX = PREC == 2 ? DEC_YMAX32 : DEC_YMAX;
    constexpr int XOR = RT <= 2 ? 1 : 2;  // lane distance of a row's first two parts
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[DEC_WARPS * DEC_STAGES];
    constexpr int QP = D + 16;  // q' of a row: its quarters 4 floats further apart (their lanes read at once)
    __shared__ float s_sv[D], s_zv[D];
    __shared__ int s_zc[D];
    // q' and the query fragments (as each lane of a warp holds them).  With one column tile, where four CTAs share an SM,
    // they lie in the last stages of the warps' rings, which no copy uses before the first turn.
    constexpr bool IN_RING = NT == 1;
    constexpr int FR = KP::N / DEC_WARPS;  // fragments that a warp makes
    static_assert(!IN_RING || FR * 128 + (S::ROWS + DEC_WARPS - 1) / DEC_WARPS * QP * 4 <= S::STAGE, "spare stage");
    __shared__ __align__(16) float s_q[IN_RING ? 4 : S::ROWS * QP];
    __shared__ uint32_t s_qf[IN_RING ? 1 : NT * KP::N * 32];
    auto spare = [&](int w) { return smem + (w * DEC_STAGES + DEC_STAGES - 1) * S::STAGE; };
    auto q_row = [&](int r) {
        return IN_RING ? reinterpret_cast<float *>(spare(r % DEC_WARPS) + FR * 128) + r / DEC_WARPS * QP : s_q + r * QP;
    };
    auto fragment = [&](int nt, int i) {
        return IN_RING ? reinterpret_cast<uint32_t *>(spare(i / FR)) + i % FR * 32 : s_qf + (nt * KP::N + i) * 32;
    };
    __shared__ __align__(16) uint8_t s_ref[S::RB];
    __shared__ float s_fac[S::ROWS][32], s_max[S::ROWS], s_inv[S::ROWS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, tq = lane & 3;
    const Paged &p = a.p;
    const int split = blockIdx.x % a.splits;
    const int bh = blockIdx.x / a.splits, b = bh / a.H, h = bh % a.H;
    // what does not hang on the sequence is asked for first: a CTA's start is a chain of loads
    const bool channel = tid < D;  // the thread's channel is tid
    const int ck = channel ? cluster_of(a.kt.ck, h * D + tid, a.kt.g, p.err) : 0;
    const int cv = channel ? cluster_of(a.kt.cv, h * D + tid, a.kt.g, p.err) : 0;
    int s0, n, L;
    if (!paged_sequence(p, b, s0, n, L)) return;
    const int rows = n * a.G;  // (token, head of the group), at most S::ROWS (the launcher's choice from max_q)
    if (rows <= 0) return;
    const int tiles = (L + DEC_TILE - 1) / DEC_TILE;
    const int stride = a.splits * DEC_WARPS, first = split * DEC_WARPS + warp;
    const int count = first < tiles ? (tiles - first - 1) / stride + 1 : 0;  // tiles of this warp

    // ---- the warp's ring ----
    const uint32_t ring = smem_u32(smem) + warp * DEC_STAGES * S::STAGE, bar0 = smem_u32(bars) + warp * DEC_STAGES * 8;
    if (lane == 0) {
        for (int s = 0; s < DEC_STAGES; ++s) mbar_init(bar0 + 8 * s, 1);
        fence_mbar_init();
    }
    __syncwarp();
    const bool small = p.shift == 4;  // pages of 16: a tile is two of them
    const int last_page = (L - 1) >> p.shift;
    int ids0 = 0, ids1 = 0;  // page ids of the 32 tiles from the last multiple of 32 on, one to a lane
    auto issue = [&](int i) {  // the i-th tile of the warp, called for i = 0, 1, ... in order
        if ((i & 31) == 0 && i + lane < count) {
            const int pg = ((first + (i + lane) * stride) * DEC_TILE) >> p.shift;
            ids0 = max(paged_page(p, b, pg), 0);
            ids1 = small && pg + 1 <= last_page ? max(paged_page(p, b, pg + 1), 0) : -1;
        }
        const int id0 = __shfl_sync(FULL, ids0, i & 31);
        const int id1 = small ? __shfl_sync(FULL, ids1, i & 31) : -1;
        if (lane == 0) {
            const int s = i % DEC_STAGES;
            const uint32_t dst = ring + s * S::STAGE, bar = bar0 + 8 * s;
            const int slot = ((first + i * stride) * DEC_TILE) & ((1 << p.shift) - 1);
            const int64_t o0 = (paged_row(id0, a.H, h, p.shift) + slot) * S::RB;
            const uint32_t bytes = small ? S::TILE / 2 : S::TILE;
            mbar_expect_tx(bar, id1 >= 0 ? 4 * bytes : 2 * bytes);
            bulk_g2s(dst, a.kq + o0, bytes, bar);
            bulk_g2s(dst + S::TILE, a.vq + o0, bytes, bar);
            if (id1 >= 0) {
                const int64_t o1 = paged_row(id1, a.H, h, p.shift) * S::RB;
                bulk_g2s(dst + bytes, a.kq + o1, bytes, bar);
                bulk_g2s(dst + S::TILE + bytes, a.vq + o1, bytes, bar);
            }
        }
    };
    int issued = 0;
    for (; issued < DEC_STAGES - 1 && issued < count; ++issued) issue(issued);

    // ---- q' = q s of the rows in fp32, position 0's codes, then the query fragments ----
    if (channel) {
        const float sk = a.kt.sk[ck];
        float q[S::ROWS];
#pragma unroll
        for (int r = 0; r < S::ROWS; ++r) {
            const int tok = r / a.G, j = r - tok * a.G;
            q[r] = r < rows ? load_elem(a.q, a.dtype, (int64_t)(s0 + tok) * a.q_stride + (int64_t)(h * a.G + j) * D + tid) : 0.f;
        }
        s_sv[tid] = a.kt.sv[cv];
        const int zv = a.kt.zv[cv], zc = PREC == 2 ? zero_code(zv, (1 << BITS) - 1) : 0;
        s_zv[tid] = (float)(zv - zc);
        s_zc[tid] = zc;
#pragma unroll
        for (int r = 0; r < S::ROWS; ++r) q_row(r)[tid + tid / (D / 4) * 4] = q[r] * sk;
    }
    if (L > 0 && tid < S::RB / 4)
        reinterpret_cast<uint32_t *>(s_ref)[tid] =
            __ldg(reinterpret_cast<const uint32_t *>(a.kq + paged_row(max(paged_page(p, b, 0), 0), a.H, h, p.shift) * S::RB) + tid);
    __syncthreads();
    // Column gq of tile nt: the lane needs the channels of its quarter in the order of the K pairs.  All warps hold the same
    // fragments; each makes a share of them.
    float cx[NT][E];  // base-2 scores of the lane's columns = cx * S
    int vis[NT][E];   // their visible positions (none in a column that holds no row)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float *v = q_row(nt * RT + S::row(gq)) + tq * (D / 4 + 4);
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < D / 4; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(v + i);
            m = fmaxf(fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y))), fmaxf(fabsf(f.z), fabsf(f.w)));
        }
        m = fmaxf(m, __shfl_xor_sync(FULL, m, 1));
        m = fmaxf(m, __shfl_xor_sync(FULL, m, 2));
        int ex = 0;
        if (m > 0.f && m < INFINITY) frexpf(m, &ex);  // m < 2^ex
        ex = max(ex, -100);
        const int grid = PREC ? 11 : 15;  // largest |q'| in [2^(grid - 1), 2^grid)
        const float up = S::used(gq) ? __uint_as_float((uint32_t)(127 + grid - ex) << 23) : 0.f;  // 2^(grid - ex)
#pragma unroll
        for (int i = 0; i < KP::N; ++i) {
            if (i / FR != warp) continue;
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float f = v[KP::code(i, e)] * up;
                if (PREC) {  // part j: the integer nearest to what the parts before it leave, times 2^(11 j)
                    float g = rintf(f);
#pragma unroll
                    for (int j = 1; j < S::PARTS; ++j)
                        if (j <= S::part(gq)) {
                            f = (f - g) * 2048.f;
                            g = rintf(f);
                        }
                    f = g;
                }
                w[e] = f * (1.f / (float)(1 << KP::pos(i, e)));
            }
            fragment(nt, i)[lane] = half2_bits(w[0], w[1]);
        }
        const float c = ldexpf(a.scale * LOG2E, ex - grid + (PREC ? 10 : 24));
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int col = 2 * tq + e, r = nt * RT + S::row(col);
            cx[nt][e] = __shfl_sync(FULL, c, 4 * col);
            vis[nt][e] = S::used(col) && r < rows ? L - n + r / a.G + 1 : 0;
        }
    }
    __syncthreads();
    uint32_t qf[NT][KP::N];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < KP::N; ++i) qf[nt][i] = fragment(nt, i)[lane];
    if (IN_RING) {  // read by all: the stages may be filled, by copies that come after these stores and loads (another proxy's)
        fence_proxy_async_smem();
        __syncthreads();
    }

    // Scores are taken relative to position 0's, subtracted in the (exact) sums of each part: what is left has the size
    // of the scores' spread, while q' code alone carries the channels' means times q.
    float xr[NT][4];  // [2] and [3] equal [0] and [1]
    {
        uint32_t kr[KP::N];
        KP::load(s_ref, tq, kr);
        if (PREC) {
#pragma unroll
            for (int j = 0; j < KP::N; ++j) kr[j] = code_up(kr[j]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) xr[nt][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                mma_16816(xr[nt], kr[2 * ks], kr[2 * ks], kr[2 * ks + 1], kr[2 * ks + 1], qf[nt][2 * ks], qf[nt][2 * ks + 1]);
        }
    }

    float o[D / 16][NT][4];  // sums over the warp's positions: channels 2i, 2i + 1 of the lane's D / 8, two columns
    float m[NT][E], off[NT][E], l[NT][E];  // reference of the exponents, PSHIFT - m, sum
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            m[nt][e] = -1e30f;
            off[nt][e] = vis[nt][e] > 0 ? 1e30f : -INFINITY;
            l[nt][e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
    }
    uint32_t vc[PREC == 2 ? VC::N : 1];  // what is taken off V's codes
    if constexpr (PREC == 2) {
#pragma unroll
        for (int j = 0; j < VC::N; ++j) {
            const float c = code_offset(s_zc[gq * (D / 8) + j], VC::pos(j));
            vc[j] = half2_bits(c, c);
        }
    }
    // position of MMA row k (0-15) of a block: k with its low bits arranged so that the rows that the lanes of one
    // shared-memory access read are neighbours, for K (rows gq) and for V (k = 2 tq, ...) alike
    const int prow = gq ^ ((gq >> 1) & 1);
    const int v0 = 2 * tq + (tq & 1), v1 = v0 ^ 1;
    const int part = S::part(2 * tq);  // of the lane's columns
    const bool head = part == 0;       // the lane's columns are the rows' first (or only) parts
    const float second = part == 1 ? -1.f : 0.f;  // a weight's second part: less its first
    const float part_scale = part == 0 ? 1.f : part == 1 ? 0x1p-11f : part == 2 ? 0x1p-22f : 0.f;

    bool ok = true;
    for (int i = 0; i < count; ++i) {
        if (issued < count) issue(issued++);
        const int s = i % DEC_STAGES;
        ok = __all_sync(FULL, mbar_wait_bounded(bar0 + 8 * s, (i / DEC_STAGES) & 1, p.err));
        if (!ok) break;
        const int pos0 = (first + i * stride) * DEC_TILE;
        const uint8_t *kst = smem + (warp * DEC_STAGES + s) * S::STAGE, *vst = kst + S::TILE;
        float x[2][NT][4];
#pragma unroll
        for (int bk = 0; bk < 2; ++bk) {
            uint32_t ka[KP::N], kb[KP::N];
            KP::load(kst + (16 * bk + prow) * S::RB, tq, ka);
            KP::load(kst + (16 * bk + prow + 8) * S::RB, tq, kb);
            if (PREC) {
#pragma unroll
                for (int j = 0; j < KP::N; ++j) ka[j] = code_up(ka[j]), kb[j] = code_up(kb[j]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[bk][nt][e] = -xr[nt][e];
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_16816(x[bk][nt], ka[2 * ks], kb[2 * ks], ka[2 * ks + 1], kb[2 * ks + 1], qf[nt][2 * ks],
                              qf[nt][2 * ks + 1]);
                if (PREC) {  // the parts' sum, in every lane of the row
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            float &v = x[bk][nt][2 * f + e];
                            v *= part_scale;
                            v += __shfl_xor_sync(FULL, v, XOR);
                            if (RT <= 2) v += __shfl_xor_sync(FULL, v, 2);
                        }
                }
            }
        }
        if (a.scores != nullptr && head) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int r = nt * RT + S::row(2 * tq + e);
                    if (r >= rows || !S::used(2 * tq + e)) continue;
                    const int tok = r / a.G, j = r - tok * a.G;
                    float *dst = a.scores + ((int64_t)(s0 + tok) * a.Hq + h * a.G + j) * p.max_len;
#pragma unroll
                    for (int bk = 0; bk < 2; ++bk)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const int pos = pos0 + 16 * bk + prow + 8 * f;
                            if (pos < L) dst[pos] = x[bk][nt][2 * f + e] * cx[nt][e];
                        }
                }
        }
        // exponents against the reference m: y = x - m + PSHIFT, -inf where the row does not see the position.
        // m only has to keep 2^y inside fp16; it moves when some y passes YMAX, seldom after the first tile.
        const bool whole = pos0 + DEC_TILE <= L - n + 1;  // every row sees the whole tile
        float y[2][NT][2][E];
        auto hide = [&]() {
            if (whole) return;
#pragma unroll
            for (int bk = 0; bk < 2; ++bk)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if (pos0 + 16 * bk + prow + 8 * f >= vis[nt][e]) y[bk][nt][f][e] = -INFINITY;
        };
        float top = -INFINITY;
#pragma unroll
        for (int bk = 0; bk < 2; ++bk)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int e = 0; e < E; ++e) y[bk][nt][f][e] = fmaf(x[bk][nt][2 * f + e], cx[nt][e], off[nt][e]);
        hide();
#pragma unroll
        for (int bk = 0; bk < 2; ++bk)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < E; ++e) top = max3f(top, y[bk][nt][0][e], y[bk][nt][1][e]);
        if (__any_sync(FULL, top > YMAX)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float mn = m[nt][e];
#pragma unroll
                    for (int bk = 0; bk < 2; ++bk)
#pragma unroll
                        for (int f = 0; f < 2; ++f)
                            if (pos0 + 16 * bk + prow + 8 * f < vis[nt][e]) mn = fmaxf(mn, x[bk][nt][2 * f + e] * cx[nt][e]);
#pragma unroll
                    for (int f = 4; f < 32; f <<= 1) mn = fmaxf(mn, __shfl_xor_sync(FULL, mn, f));
                    if (vis[nt][e] > 0 && mn > -1e30f) {
                        mn = ceilf(mn);  // an integer: PSHIFT - m is exact, and so is the factor between two references
                        const float r = ex2(m[nt][e] - mn);
                        m[nt][e] = mn;
                        off[nt][e] = (float)PSHIFT - mn;
                        l[nt][e] *= r;
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            o[c][nt][e] *= r;
                            o[c][nt][2 + e] *= r;
                        }
                    }
#pragma unroll
                    for (int bk = 0; bk < 2; ++bk)
#pragma unroll
                        for (int f = 0; f < 2; ++f) y[bk][nt][f][e] = fmaf(x[bk][nt][2 * f + e], cx[nt][e], off[nt][e]);
                }
            hide();
        }
        // weights, then O += V^T w^T block by block
#pragma unroll
        for (int bk = 0; bk < 2; ++bk) {
            uint32_t w[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    float pv[2] = {0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < E; ++e) pv[e] = ex2(y[bk][nt][f][e]);
                    uint32_t hw = half2_bits(pv[0], pv[1]);
                    const float2 r2 = __half22float2(*reinterpret_cast<const __half2 *>(&hw));
                    if (PREC) {  // two parts, in the columns of q's first two (what is in the others is not used)
#pragma unroll
                        for (int e = 0; e < E; ++e) l[nt][e] += pv[e];
                        hw = half2_bits(fmaf(r2.x, second, pv[0]), fmaf(r2.y, second, pv[1]));
                    } else {  // the rounded weights are summed: numerator and denominator hold the same ones
                        l[nt][0] += r2.x;
                        if (E == 2) l[nt][E - 1] += r2.y;
                    }
                    w[nt][f] = mat_trans(hw);
                }
            uint32_t ra[VC::NW], rc[VC::NW], xa[VC::N], xb[VC::N];
            VC::load(vst + (16 * bk + v0) * S::RB, gq, ra);
            VC::load(vst + (16 * bk + v1) * S::RB, gq, rc);
            VC::join(ra, rc, xa);
            VC::load(vst + (16 * bk + v0 + 8) * S::RB, gq, ra);
            VC::load(vst + (16 * bk + v1 + 8) * S::RB, gq, rc);
            VC::join(ra, rc, xb);
            if constexpr (PREC == 2) {
#pragma unroll
                for (int j = 0; j < VC::N; ++j) xa[j] = code_up_plus(xa[j], vc[j]), xb[j] = code_up_plus(xb[j], vc[j]);
            }
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (PREC == 2) {
                        // The tensor core cuts its sums off at the accumulator's last bit, every one to the same side (1.3e-6
                        // of the result after 8540 positions, measured): over the blocks they are added and rounded here.
                        float t[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_16816(t, xa[2 * c], xa[2 * c + 1], xb[2 * c], xb[2 * c + 1], w[nt][0], w[nt][1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[c][nt][e] += t[e];
                    } else {
                        mma_16816(o[c][nt], xa[2 * c], xa[2 * c + 1], xb[2 * c], xb[2 * c + 1], w[nt][0], w[nt][1]);
                    }
                }
        }
        fence_proxy_async_smem();
        __syncwarp();  // the stage has been read (its values went into the MMAs above): the next turn's copy may fill it
    }
    if (!ok)  // a wait ran out: no copy may be in flight into this CTA's memory when it ends
        for (int i = max(0, issued - DEC_STAGES); i < issued; ++i)
            mbar_wait_bounded(bar0 + 8 * (i % DEC_STAGES), (i / DEC_STAGES) & 1, p.err);

    // ---- join the warps ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int f = 4; f < 32; f <<= 1) l[nt][e] += __shfl_xor_sync(FULL, l[nt][e], f);
    __syncthreads();  // every warp is done with its ring
    float *js = reinterpret_cast<float *>(smem);            // [warp][row][D]
    float *jm = js + DEC_WARPS * S::ROWS * D;               // [warp][row]
    float *jl = jm + DEC_WARPS * S::ROWS;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int r = nt * RT + S::row(2 * tq + e);
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    float v = o[c][nt][2 * f + e];
                    if (PREC) v += __shfl_xor_sync(FULL, v, XOR);
                    // the codes' power of two and the weights' 2^PSHIFT
                    v *= (float)(1 << ((PREC == 2 ? 10 : 24) - VC::pos(2 * c + f))) * (1.f / (float)(1 << PSHIFT));
                    if (head) js[(warp * S::ROWS + r) * D + gq * (D / 8) + 2 * c + f] = v;
                }
            if (gq == 0 && head) {
                jm[warp * S::ROWS + r] = l[nt][e] == 0.f ? -INFINITY : m[nt][e];
                jl[warp * S::ROWS + r] = l[nt][e] * (1.f / (float)(1 << PSHIFT));
            }
        }
    __syncthreads();
    auto row_of = [&](int r) { return (int64_t)(s0 + r / a.G) * a.Hq + h * a.G + r % a.G; };
    if (a.part != nullptr) {  // more parts than a cluster has CTAs: a second kernel joins them
        for (int i = tid; i < rows * D; i += DEC_THREADS) {
            const int r = i / D, d = i - r * D;
            const int64_t row = row_of(r);
            float mt = -INFINITY, lt = 0.f, v = 0.f;
#pragma unroll
            for (int w = 0; w < DEC_WARPS; ++w) mt = fmaxf(mt, jm[w * S::ROWS + r]);
#pragma unroll
            for (int w = 0; w < DEC_WARPS; ++w) {
                const float mw = jm[w * S::ROWS + r];
                const float f = mw == -INFINITY ? 0.f : ex2(mw - mt);
                lt = fmaf(jl[w * S::ROWS + r], f, lt);
                v = fmaf(js[(w * S::ROWS + r) * D + d], f, v);
            }
            a.part[((int64_t)split * p.T * a.Hq + row) * D + d] = v;
            if (d == 0) {
                float *ml = a.ml + ((int64_t)split * p.T * a.Hq + row) * 2;
                ml[0] = mt;
                ml[1] = lt;
            }
        }
        return;
    }
    // the parts are the CTAs of this cluster: every CTA takes the rows' maxima and sums over all their warps, its share of
    // the outputs, and (running sums) the positions that it scored itself
    cg::cluster_group cluster = cg::this_cluster();
    const int all = a.splits * DEC_WARPS;  // warps of the cluster
    cluster.sync();
    for (int r = warp; r < rows; r += DEC_WARPS) {
        const float *om = cluster.map_shared_rank(jm, min(lane / DEC_WARPS, a.splits - 1));
        const float *ol = om + (jl - jm);
        const float mw = lane < all ? om[lane % DEC_WARPS * S::ROWS + r] : -INFINITY;
        float mt = mw;
        for (int f = 16; f > 0; f >>= 1) mt = fmaxf(mt, __shfl_xor_sync(FULL, mt, f));
        const float f = mw == -INFINITY ? 0.f : ex2(mw - mt);
        float lt = lane < all ? ol[lane % DEC_WARPS * S::ROWS + r] * f : 0.f;
        for (int o = 16; o > 0; o >>= 1) lt += __shfl_xor_sync(FULL, lt, o);
        s_fac[r][lane] = f;
        if (lane == 0) s_max[r] = mt, s_inv[r] = mt == -INFINITY ? 0.f : 1.f / lt;
    }
    __syncthreads();
    for (int i = split * DEC_THREADS + tid; i < rows * D; i += a.splits * DEC_THREADS) {
        const int r = i / D, d = i - r * D;
        float v = 0.f;
        for (int c = 0; c < a.splits; ++c) {
            const float *os = cluster.map_shared_rank(js, c);
#pragma unroll
            for (int w = 0; w < DEC_WARPS; ++w) v = fmaf(os[(w * S::ROWS + r) * D + d], s_fac[r][c * DEC_WARPS + w], v);
        }
        store_elem(a.out, a.dtype, row_of(r) * D + d, s_max[r] == -INFINITY ? 0.f : s_sv[d] * (v * s_inv[r] - s_zv[d]));
    }
    if (a.weights != nullptr) {
        constexpr int U = 8;  // tiles whose loads are in flight together
        for (int i0 = 0; i0 < count; i0 += U) {
            int pos[U];
            float *at[U], old[U], w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                pos[u] = i0 + u < count ? (first + (i0 + u) * stride) * DEC_TILE + lane : L;
                const int page = pos[u] < L ? paged_page(p, b, pos[u] >> p.shift) : -1;
                at[u] = page < 0 ? nullptr : a.weights + paged_row(page, a.H, h, p.shift) + (pos[u] & ((1 << p.shift) - 1));
                w[u] = 0.f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) old[u] = at[u] ? *at[u] : 0.f;
            for (int r = 0; r < rows; ++r) {
                const float *x = a.scores + row_of(r) * p.max_len;
                const int seen = L - n + r / a.G + 1;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (at[u] && pos[u] < seen) w[u] = fmaf(ex2(x[pos[u]] - s_max[r]), s_inv[r], w[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (at[u]) *at[u] = old[u] + w[u];
        }
    }
    cluster.sync();  // the others may still be reading this CTA's shared memory
}

// Joins the parts of every row, a CTA to a row.
constexpr int CMB_THREADS = 128;

template <int D>
__global__ void __launch_bounds__(CMB_THREADS)
    paged_combine_kernel(const PagedAttnDev a)
{
    extern __shared__ float s_f[];  // a factor per part
    const Paged &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t R = p.T * a.Hq, row = blockIdx.x;
    const int b = paged_row_sequence(p, row / a.Hq);
    int s0, n, L;
    if (b < 0 || !paged_sequence(p, b, s0, n, L)) return;
    float mt = -INFINITY, lt = 0.f;  // the same in every warp
    for (int s = lane; s < a.splits; s += 32) mt = fmaxf(mt, a.ml[(s * R + row) * 2]);
    for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(FULL, mt, o));
    for (int s = lane; s < a.splits; s += 32) {
        const float ms = a.ml[(s * R + row) * 2];
        if (ms != -INFINITY) lt = fmaf(a.ml[(s * R + row) * 2 + 1], ex2(ms - mt), lt);
    }
    for (int o = 16; o > 0; o >>= 1) lt += __shfl_xor_sync(FULL, lt, o);
    for (int s = tid; s < a.splits; s += CMB_THREADS) {
        const float ms = a.ml[(s * R + row) * 2];
        s_f[s] = ms == -INFINITY ? 0.f : ex2(ms - mt) / lt;
    }
    __syncthreads();
    if (a.stat != nullptr && tid == 0) {
        a.stat[2 * row] = mt == -INFINITY ? 0.f : mt;
        a.stat[2 * row + 1] = mt == -INFINITY ? 0.f : 1.f / lt;
    }
    const int h = (int)(row % a.Hq) / a.G;
    for (int d = tid; d < D; d += CMB_THREADS) {
        float v = 0.f;
#pragma unroll 8
        for (int s = 0; s < a.splits; ++s) v = fmaf(a.part[(s * R + row) * D + d], s_f[s], v);
        const int k = cluster_of(a.kt.cv, h * D + d, a.kt.g, p.err);
        store_elem(a.out, a.dtype, row * D + d, mt == -INFINITY ? 0.f : a.kt.sv[k] * (v - (float)(a.kt.zv[k] - zero_code(a.kt.zv[k], a.centred))));
    }
}

// ---- launch ----------------------------------------------------------------------------------------------
namespace {
struct DecPlan {
    int prec, rt, nt, splits;
    bool second;  // a second kernel joins the parts
};
constexpr int DEC_MAX_SPLITS = 64, DEC_CLUSTER = 8;
DecPlan dec_plan(int Hq, int H, int dtype, int B, int max_q, int max_len, int weights, int num_sms)
{
    DecPlan pl;
    const int64_t rows = (int64_t)max_q * (Hq / H);
    pl.prec = dtype == RPTQ_F32 ? 2 : weights || dtype == RPTQ_F16 ? 1 : 0;
    pl.rt = rows == 1 ? 1 : weights || pl.prec == 2 ? 2 : pl.prec == 1 ? 4 : 8;
    pl.nt = rows <= pl.rt ? 1 : rows <= 2 * pl.rt ? 2 : 4;
    // Parts: about DEC_CTAS_SM CTAs to an SM in all, each warp at least a tile.  Up to DEC_CLUSTER (always, where running sums are kept)
    // they are a cluster, which joins itself; more leave their results to a second kernel.
    const int64_t units = (int64_t)B * H, tiles = (max_len + DEC_TILE - 1) / DEC_TILE;
    const int64_t want = std::min((DEC_CTAS_SM * num_sms + units / 2) / units, tiles / DEC_WARPS);
    if (want > DEC_CLUSTER && !weights) {
        pl.splits = (int)std::min<int64_t>(want, DEC_MAX_SPLITS);
    } else {
        pl.splits = 1;
        while (pl.splits < want && pl.splits < DEC_CLUSTER) pl.splits *= 2;
    }
    pl.second = pl.splits > DEC_CLUSTER;
    return pl;
}
}  // namespace

// at most four column tiles: 8 rows in three parts, 16 in two, 32 in one
bool paged_decode_takes(int Hq, int H, int D, int dtype, int max_q, int weights)
{
    if (D != 64 && D != 128) return false;
    const int64_t rows = (int64_t)max_q * (Hq / H);
    return rows <= (weights || dtype == RPTQ_F32 ? 8 : dtype == RPTQ_F16 ? 16 : 32);
}

size_t paged_decode_workspace(int64_t T, int Hq, int H, int D, int dtype, int B, int max_q, int max_len, int weights,
                              int num_sms)
{
    const DecPlan pl = dec_plan(Hq, H, dtype, B, max_q, max_len, weights, num_sms);
    size_t bytes = 0;
    if (pl.second) bytes += (size_t)pl.splits * T * Hq * (D + 2) * 4;
    if (weights) bytes += (size_t)T * Hq * max_len * 4;
    return bytes;
}

template <int BITS, int D, int RT, int NT, int PREC>
static cudaError_t launch_dec(const PagedAttnDev &d, const DecPlan &pl, int B, cudaStream_t stream)
{
    using S = DecShape<BITS, D, RT, NT, PREC>;
    auto kern = paged_decode_kernel<BITS, D, RT, NT, PREC>;
    cudaError_t e = kernel_smem((const void *)kern, S::SMEM);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((int64_t)B * d.H * pl.splits);
    if (pl.second || pl.splits == 1) {
        kern<<<grid, DEC_THREADS, S::SMEM, stream>>>(d);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(DEC_THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)pl.splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, d);
}
template <int BITS, int D, int RT, int PREC>
static cudaError_t launch_dec_prec(const PagedAttnDev &d, const DecPlan &pl, int B, cudaStream_t stream)
{
    if (pl.rt == 1) return launch_dec<BITS, D, 1, 1, PREC>(d, pl, B, stream);
    return pl.nt == 1   ? launch_dec<BITS, D, RT, 1, PREC>(d, pl, B, stream)
           : pl.nt == 2 ? launch_dec<BITS, D, RT, 2, PREC>(d, pl, B, stream)
                        : launch_dec<BITS, D, RT, 4, PREC>(d, pl, B, stream);
}
template <int BITS, int D>
static cudaError_t launch_dec_rows(const PagedAttnDev &d, const DecPlan &pl, int B, cudaStream_t stream)
{
    if (pl.prec == 2) return launch_dec_prec<BITS, D, 2, 2>(d, pl, B, stream);
    if (pl.prec == 0) return launch_dec_prec<BITS, D, 8, 0>(d, pl, B, stream);
    return d.weights ? launch_dec_prec<BITS, D, 2, 1>(d, pl, B, stream) : launch_dec_prec<BITS, D, 4, 1>(d, pl, B, stream);
}

cudaError_t launch_paged_decode(const PagedAttnArgs &a)
{
    const DecPlan pl = dec_plan(a.Hq, a.H, a.dtype, a.B, a.max_q, a.max_len, a.weights != nullptr, a.num_sms);
    PagedAttnDev d{};
    d.p = Paged{a.start, a.lens, a.table, a.B, a.max_pages, a.shift, a.n_pages, a.T, a.max_q, a.max_len, a.err};
    d.q = a.q, d.out = a.out, d.dtype = a.dtype, d.Hq = a.Hq, d.H = a.H, d.G = a.Hq / a.H, d.q_stride = a.q_stride;
    d.kq = a.kq, d.vq = a.vq, d.kt = a.kt, d.scale = a.scale, d.weights = a.weights, d.splits = pl.splits;
    d.centred = pl.prec == 2 ? (1 << a.bits) - 1 : 0;
    if (a.weights) d.scores = static_cast<float *>(a.ws);
    if (pl.second) {
        d.part = static_cast<float *>(a.ws);
        d.ml = d.part + (int64_t)pl.splits * a.T * a.Hq * a.D;
    }
    cudaError_t e = a.bits == 4 ? (a.D == 128 ? launch_dec_rows<4, 128>(d, pl, a.B, a.stream) : launch_dec_rows<4, 64>(d, pl, a.B, a.stream))
                                : (a.D == 128 ? launch_dec_rows<3, 128>(d, pl, a.B, a.stream) : launch_dec_rows<3, 64>(d, pl, a.B, a.stream));
    if (e != cudaSuccess || !pl.second) return e;
    return launch_paged_combine(d, a.D, a.stream);
}

cudaError_t launch_paged_combine(const PagedAttnDev &d, int D, cudaStream_t stream)
{
    const unsigned grid = (unsigned)(d.p.T * d.Hq);
    const size_t smem = (size_t)d.splits * 4;
    if (D == 128)
        paged_combine_kernel<128><<<grid, CMB_THREADS, smem, stream>>>(d);
    else
        paged_combine_kernel<64><<<grid, CMB_THREADS, smem, stream>>>(d);
    return cudaGetLastError();
}

}  // namespace rptq
