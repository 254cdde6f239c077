// kv_paged.cu -- the paged packed K/V cache: tokens quantized into pages, read back, and evicted.
//
// RPTQ article (基于重排序的新量化方法RPTQ…), results paragraph (the K and V caches quantized per
// cluster) and closing memory paragraph (the cache dominates memory at large batch x sequence): the
// same codes as the dense cache's, in pages, so that sequences of unequal length share one pool
// (kv_paged.cuh has the layout).
#include <cooperative_groups.h>

#include <algorithm>

#include "kv_codec.cuh"
#include "kv_paged.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace rptq {

// ---- append and read-back ------------------------------------------------------------------------
// A thread owns 8 consecutive channels, whose coefficients stay in registers, and walks the rows of
// its CTA's chunk of the batch; blockIdx.y is the slab of blockDim.x * 8 channels, blockIdx.z the
// tensor.  Where each row of the chunk lives is looked up once per CTA.  Both directions move each
// byte once and are bound by HBM at large batches and by the launch at small ones (calls one behind another, each on other inputs:
// 9 prompts of about 1100 tokens, 96 heads of 128, 3 bits: append and read-back 219 us, 4.7 TB/s; 8 x 2048 positions read back,
// K and V: 179 us, 4.85 TB/s).
constexpr int PG_THREADS = 256;
constexpr int PG_ROWS = 256;  // most rows of a CTA's chunk
constexpr int PG_UNROLL = 4;  // 16-byte loads (words, for the read-back) of a step, the next step's issued before it

// Four lanes' 24-bit groups <-> the three 32-bit words they fill (lane j of the four holds word j < 3).
__device__ __forceinline__ uint32_t pack_a3_words(uint32_t grp, int lane)
{
    const uint32_t next = __shfl_down_sync(FULL, grp, 1);
    const int j = lane & 3;
    return (grp >> (8 * j)) | (next << (24 - 8 * j));
}
__device__ __forceinline__ uint32_t unpack_a3_words(uint32_t w, int lane)
{
    const int j = lane & 3, base = lane & ~3;
    const uint32_t lo = __shfl_sync(FULL, w, base + (j == 3 ? 2 : max(j - 1, 0)));
    const uint32_t hi = __shfl_sync(FULL, w, base + min(j, 2));
    // group j is bits 24j .. 24j + 23 of the 96: words (0), (0, 1), (1, 2), (2); what is above its 24 bits is not its own
    return __funnelshift_r(lo, hi, (32 - 8 * j) & 31);
}

template <typename T, int BITS>
__global__ void __launch_bounds__(PG_THREADS, 2)
    kv_paged_append_kernel(KvTensors t, Paged p, int64_t row_stride, int H, int D, int g, int rows_per_cta,
                           float *__restrict__ weights)
{
    constexpr int VEC = Elem<T>::VEC, NLD = 8 / VEC;
    constexpr int U = PG_UNROLL / NLD;  // rows of a step
    __shared__ int64_t s_row[PG_ROWS];  // byte of head 0's row of each position; -1: none
    const int tid = threadIdx.x, lane = tid & 31;
    const T *src = static_cast<const T *>(t.src[blockIdx.z]);
    if (src == nullptr) return;
    uint8_t *dst = t.dst[blockIdx.z];
    const int64_t t0 = (int64_t)blockIdx.x * rows_per_cta;
    const int rows = (int)min((int64_t)rows_per_cta, p.T - t0);
    for (int r = tid; r < rows; r += blockDim.x) {
        int page = -1, slot = 0;
        const int b = paged_row_sequence(p, t0 + r);
        int s0, n, L;
        if (b >= 0 && paged_sequence(p, b, s0, n, L)) {
            const int pos = L - n + (int)(t0 + r - s0);
            if (pos >= 0) {
                page = paged_page(p, b, pos >> p.shift);
                slot = pos & ((1 << p.shift) - 1);
            }
        }
        s_row[r] = page < 0 ? -1 : (paged_row(page, H, 0, p.shift) + slot) * (D * BITS / 8);
    }
    const int c0 = (blockIdx.y * blockDim.x + tid) * 8;
    const bool live = c0 < H * D;
    const int c = live ? c0 : 0, h = c / D, d0 = c - h * D;
    KvCoef<BITS, 8> cf;
    cf.load(t.cl[blockIdx.z], t.sc[blockIdx.z], t.zp[blockIdx.z], c, g, p.err);
    __syncthreads();
    const int rb = D * BITS / 8;
    const T *col = src + t0 * row_stride + c;  // of the next rows to load
    // the thread's word of a row; of the four lanes that share 96 bits, three store
    const bool mine = live && (BITS == 4 || (lane & 3) < 3);
    uint8_t *word = dst + ((int64_t)h << p.shift) * rb + (BITS == 4 ? d0 / 2 : (d0 & ~31) * 3 / 8 + (lane & 3) * 4);
    const bool zeroes = weights != nullptr && blockIdx.z == 0 && live && d0 == 0;
    uint4 x[U][NLD];  // the next U rows, loaded while the U before them are quantized
    auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int l = 0; l < NLD; ++l)
                x[u][l] = i0 + u < rows ? ldg_stream(col + u * row_stride + l * VEC) : make_uint4(0, 0, 0, 0);
        col += U * row_stride;
    };
    load(0);
    for (int i0 = 0; i0 < rows; i0 += U) {
        uint4 y[U][NLD];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int l = 0; l < NLD; ++l) y[u][l] = x[u][l];
        if (i0 + U < rows) load(i0 + U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            if (i >= rows) break;
            uint32_t grp[1];
            kv_quant_row<T, BITS, 8>(y[u], cf, grp);
            const uint32_t w = BITS == 4 ? grp[0] : pack_a3_words(grp[0], lane);
            const int64_t row = s_row[i];
            if (!mine || row < 0) continue;
            *reinterpret_cast<uint32_t *>(word + row) = w;
            if (zeroes) weights[row / rb + ((int64_t)h << p.shift)] = 0.f;
        }
    }
}

template <typename T> __device__ __forceinline__ void store8(T *dst, const float (&v)[8]);
template <> __device__ __forceinline__ void store8<float>(float *dst, const float (&v)[8])
{
    __stcs(reinterpret_cast<float4 *>(dst), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4 *>(dst) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
template <> __device__ __forceinline__ void store8<__half>(__half *dst, const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(w[0], w[1], w[2], w[3]));
}
template <> __device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16 *dst, const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(w[0], w[1], w[2], w[3]));
}

template <typename T, int BITS>
__global__ void __launch_bounds__(PG_THREADS)
    kv_paged_dequant_kernel(const uint8_t *__restrict__ pages, Paged p, int H, int D, const int32_t *__restrict__ cluster,
                            const float *__restrict__ scale, const int32_t *__restrict__ zero, int g, int rows_per_cta,
                            T *__restrict__ out)
{
    constexpr uint32_t MASK = (1u << BITS) - 1u;
    __shared__ int64_t s_row[PG_ROWS];  // byte of head 0's row of each position; -1: none
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t t0 = (int64_t)blockIdx.x * rows_per_cta;
    const int rows = (int)min((int64_t)rows_per_cta, p.T - t0);
    for (int r = tid; r < rows; r += blockDim.x) {
        int page = -1, slot = 0;
        const int b = paged_row_sequence(p, t0 + r);
        if (b >= 0) {  // p.lens: the first position read of each sequence
            const int64_t pos = (int64_t)p.lens[b] + (t0 + r - p.start[b]);
            if (pos >= 0 && pos < p.max_len) {
                page = paged_page(p, b, (int)(pos >> p.shift));
                slot = (int)pos & ((1 << p.shift) - 1);
            } else {
                raise_error(p.err, RPTQ_DEVERR_RANGE);
            }
        }
        s_row[r] = page < 0 ? -1 : (paged_row(page, H, 0, p.shift) + slot) * (D * BITS / 8);
    }
    const int c0 = (blockIdx.y * blockDim.x + tid) * 8;
    const bool live = c0 < H * D;
    const int c = live ? c0 : 0, h = c / D, d0 = c - h * D;
    auto cluster_at = [&](int j) {
        const int k = cluster[c + j];
        return k >= 0 && k < g ? k : 0;
    };
    f32x2 s2[4], nz2[4];
    bool near = true;  // every zero point small enough for the exact difference below
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        int z[2];
        float s[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int k = cluster[c + 2 * j + e];
            if (k < 0 || k >= g) raise_error(p.err, RPTQ_DEVERR_CLUSTER_ID);
            s[e] = scale[cluster_at(2 * j + e)];
            z[e] = zero[cluster_at(2 * j + e)];
            near = near && z[e] > -(1 << 22) && z[e] < (1 << 22);
        }
        s2[j] = mk2(s[0], s[1]);
        nz2[j] = mk2(-(8388608.f + (float)z[0]), -(8388608.f + (float)z[1]));
    }
    __syncthreads();
    const int rb = D * BITS / 8;
    const uint8_t *word = pages + ((int64_t)h << p.shift) * rb + (BITS == 4 ? d0 / 2 : (d0 & ~31) * 3 / 8 + min(lane & 3, 2) * 4);
    const int HD = H * D;
    T *col = out + t0 * HD + c;
    constexpr int U = PG_UNROLL;
    uint32_t x[U];  // the next U rows' words, loaded while the U before them are written
    auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = s_row[min(i0 + u, rows - 1)];
            x[u] = ldg_stream32(word + max(row, (int64_t)0));
        }
    };
    load(0);
    for (int i0 = 0; i0 < rows; i0 += U) {
        uint32_t w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = x[u];
        if (i0 + U < rows) load(i0 + U);
        if (i0 > 0) col += U * (int64_t)HD;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            if (i >= rows) break;
            const uint32_t grp = BITS == 4 ? w[u] : unpack_a3_words(w[u], lane);
            if (!live || s_row[i] < 0) continue;
            float v[8];
            if (near) {  // 2^23 + code less 2^23 + z: code - z exactly
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x2 q = mk2(__uint_as_float((grp >> (2 * BITS * j)) & MASK | 0x4B000000u),
                                        __uint_as_float((grp >> (2 * BITS * j + BITS)) & MASK | 0x4B000000u));
                    const f32x2 r = mul2(s2[j], add2(q, nz2[j]));
                    v[2 * j] = lo2(r), v[2 * j + 1] = hi2(r);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = cluster_at(j);
                    v[j] = scale[k] * (float)((int)((grp >> (BITS * j)) & MASK) - zero[k]);
                }
            }
            store8(col + u * HD, v);
        }
    }
}

// Rows of a CTA: `per_sm` CTAs to an SM, about two waves, where PG_ROWS rows are enough.  A CTA begins with the look-up of
// its channels' clusters, so few long ones (at 15300 rows of 12288 channels: 32 rows to a CTA 218 us, one wave 181, two 173).
static void paged_rows_grid(int64_t T, int C, int tensors, int num_sms, int per_sm, int *threads, int *rows, dim3 *grid)
{
    *threads = std::min(PG_THREADS, (C / 8 + 31) / 32 * 32);
    const int slabs = (C / 8 + *threads - 1) / *threads;
    const int64_t ctas = std::max(1, per_sm * num_sms / (slabs * tensors));  // in the row direction
    *rows = (int)std::max<int64_t>(1, std::min<int64_t>((T + ctas - 1) / ctas, PG_ROWS));
    *grid = dim3((unsigned)((T + *rows - 1) / *rows), (unsigned)slabs, (unsigned)tensors);
}

template <typename T>
static cudaError_t launch_paged_append_t(const PagedAppendArgs &a)
{
    const KvTensors t{{a.k, a.v}, {a.kq, a.vq}, {a.ck, a.cv}, {a.sk, a.sv}, {a.zk, a.zv}};
    const Paged p{a.start, a.lens, a.table, a.B, a.max_pages, a.shift, a.n_pages, a.T, 0x7fffffff, a.max_len, a.err};
    int threads, rows;
    dim3 grid;
    paged_rows_grid(a.T, a.H * a.D, 2, a.num_sms, 4, &threads, &rows, &grid);
    if (a.bits == 4)
        kv_paged_append_kernel<T, 4><<<grid, threads, 0, a.stream>>>(t, p, a.row_stride, a.H, a.D, a.g, rows, a.weights);
    else
        kv_paged_append_kernel<T, 3><<<grid, threads, 0, a.stream>>>(t, p, a.row_stride, a.H, a.D, a.g, rows, a.weights);
    return cudaGetLastError();
}

cudaError_t launch_paged_append(const PagedAppendArgs &a)
{
    switch (a.dtype) {
    case RPTQ_F32: return launch_paged_append_t<float>(a);
    case RPTQ_F16: return launch_paged_append_t<__half>(a);
    default: return launch_paged_append_t<__nv_bfloat16>(a);
    }
}

template <typename T>
static cudaError_t launch_paged_dequant_t(const PagedDequantArgs &a)
{
    const Paged p{a.start, a.begin, a.table, a.B, a.max_pages, a.shift, a.n_pages, a.T, 0x7fffffff, a.max_len, a.err};
    int threads, rows;
    dim3 grid;
    paged_rows_grid(a.T, a.H * a.D, 1, a.num_sms, 8, &threads, &rows, &grid);
    T *out = static_cast<T *>(a.out);
    if (a.bits == 4)
        kv_paged_dequant_kernel<T, 4><<<grid, threads, 0, a.stream>>>(a.pages, p, a.H, a.D, a.cluster, a.scale, a.zero,
                                                                      a.g, rows, out);
    else
        kv_paged_dequant_kernel<T, 3><<<grid, threads, 0, a.stream>>>(a.pages, p, a.H, a.D, a.cluster, a.scale, a.zero,
                                                                      a.g, rows, out);
    return cudaGetLastError();
}

cudaError_t launch_paged_dequant(const PagedDequantArgs &a)
{
    switch (a.out_dtype) {
    case RPTQ_F32: return launch_paged_dequant_t<float>(a);
    case RPTQ_F16: return launch_paged_dequant_t<__half>(a);
    default: return launch_paged_dequant_t<__nv_bfloat16>(a);
    }
}

// ---- eviction --------------------------------------------------------------------------------------
// One cluster of CTAs per (sequence, head): each CTA has a contiguous share of the positions, whose keys (an unsigned
// number in the weights' order) it reads once into shared memory, many loads in flight.  The key of the m-th largest
// candidate is found by four passes of an 8-bit histogram from the top byte down (a radix select), each pass summed over
// the cluster through distributed shared memory; `ties` of the candidates equal to it are kept, lowest positions
// first.  With the shares' counts exchanged every CTA writes its part of the list of kept positions.  Entry j of that
// list moves from position kept[j] >= j to j: a batch of rows is loaded by the whole cluster, then stored.  A row
// stored at j < i is never one that a later entry i reads (kept[i] >= i), so the only hazard is inside a batch, and one
// cluster barrier between its loads and stores covers it.  The bound is the latency of those steps, so few (sequence, head)
// pairs get a wide cluster.  (16 x 32 heads of about 2048 to 1024, 3 bits: 61 us, with the read-back of what is left 108; 8 heads
// of 32700 to 4096, 4 bits: 30 and 36 us.)
constexpr int EV_SMALL = 256;  // threads of a CTA where there are many
constexpr int EV_UNITS = 4;   // units of a batch per thread
constexpr int EV_LOADS = 8;   // weights of a thread in flight together
constexpr int EV_MAX_CLUSTER = 8;
constexpr int EV_KEYS = 48 * 1024;  // keys that fit a CTA's shared memory; beyond, they are read again in every pass

// Larger weight, larger key; both zeros alike; NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
    if (w != w) return 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <typename U, int EV_THREADS>
__global__ void __launch_bounds__(EV_THREADS)
    kv_paged_evict_kernel(uint8_t *__restrict__ kq, uint8_t *__restrict__ vq, float *__restrict__ weights, Paged p, int H,
                          int rb, int budget, int recent, int cached, int32_t *__restrict__ new_lens, int32_t *__restrict__ kept)
{
    constexpr int EV_WARPS = EV_THREADS / 32;
    extern __shared__ uint32_t s_key[];  // the share's keys, where `cached` of them fit
    __shared__ int hist[2][256], total[256];
    __shared__ int s_eq[EV_WARPS], s_keep[EV_WARPS], s_digit, s_need, s_bad, s_first;
    __shared__ int s_share[2];  // equal candidates, kept others of this CTA
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = blockIdx.x / CS, b = bh / H, h = bh % H;
    int32_t *list = kept + (int64_t)bh * budget;
    const int L = p.lens[b];
    const int32_t *tab = p.table + (int64_t)b * p.max_pages;
    const int pmask = (1 << p.shift) - 1;
    if (tid == 0) s_bad = 0, s_first = 0x7fffffff;
    for (int i = tid; i < 256; i += EV_THREADS) hist[0][i] = 0;
    __syncthreads();
    bool bad = L < 0 || L > p.max_len;
    if (bad && tid == 0) raise_error(p.err, RPTQ_DEVERR_RANGE);
    if (!bad && L > budget)  // an evicted sequence's pages are all checked, by every CTA, before anything moves
        for (int i = tid; i < (L + pmask) >> p.shift; i += EV_THREADS)
            if (paged_page(p, b, i) < 0) s_bad = 1;
    __syncthreads();
    bad |= s_bad != 0;
    if (h == 0 && rank == 0 && tid == 0) new_lens[b] = bad ? L : min(L, budget);
    if (bad || L <= budget) {  // the same in every CTA of the cluster
        const int n = bad ? 0 : L;
        for (int64_t j = rank * EV_THREADS + tid; j < budget; j += CS * EV_THREADS) list[j] = j < n ? (int)j : -1;
        return;
    }
    auto row_of = [&](int pos) -> int64_t { return paged_row(tab[pos >> p.shift], H, h, p.shift) + (pos & pmask); };
    const int share = ((L + CS - 1) / CS + 31) & ~31;
    const int x0 = min(L, rank * share), x1 = min(L, x0 + share);  // this CTA's positions
    const bool in_smem = share <= cached;
    if (in_smem)
        for (int i0 = x0; i0 < x1; i0 += EV_THREADS * EV_LOADS) {
            float w[EV_LOADS];
#pragma unroll
            for (int k = 0; k < EV_LOADS; ++k) {
                const int pos = i0 + k * EV_THREADS + tid;
                w[k] = pos < x1 ? weights[row_of(pos)] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < EV_LOADS; ++k) {
                const int pos = i0 + k * EV_THREADS + tid;
                if (pos < x1) s_key[pos - x0] = weight_key(w[k]);
            }
        }
    __syncthreads();
    auto key_of = [&](int pos) { return in_smem ? s_key[pos - x0] : weight_key(weights[row_of(pos)]); };
    const int cand = L - recent;  // candidates: the positions below; budget - recent of them stay
    const int c1 = min(x1, cand);
    uint32_t prefix = 0, mask = 0;
    int need = budget - recent;
    for (int sh = 24, pass = 0; sh >= 0 && need > 0; sh -= 8, ++pass) {
        int *mine = hist[pass & 1];
        for (int i0 = x0 + warp * 32; i0 < c1; i0 += EV_THREADS) {
            const int pos = i0 + lane;
            const uint32_t key = pos < c1 ? key_of(pos) : 0u;
            const bool in = pos < c1 && (key & mask) == prefix;
            const uint32_t digit = in ? (key >> sh) & 255u : 256u;
            const uint32_t same = __match_any_sync(FULL, digit);
            if (in && lane == __ffs(same) - 1) atomicAdd(&mine[digit], __popc(same));
        }
        cluster.sync();
        for (int i = tid; i < 256; i += EV_THREADS) {
            int t = 0;
            for (int r = 0; r < CS; ++r) t += cluster.map_shared_rank(mine, r)[i];
            total[i] = t;
            hist[(pass + 1) & 1][i] = 0;  // read by others in the pass before only
        }
        __syncthreads();
        if (warp == 0) {  // lane l: bins 255 - 8l .. 248 - 8l; the digit where the count from the top reaches need
            int c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += c[i] = total[255 - 8 * lane - i];
            int before = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(FULL, before, o);
                if (lane >= o) before += v;
            }
            before -= sum;
            if (before < need && before + sum >= need) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < need && before + c[i] >= need) {
                        s_digit = 255 - 8 * lane - i;
                        s_need = need - before;
                        break;
                    }
                    before += c[i];
                }
            }
        }
        __syncthreads();
        prefix |= (uint32_t)s_digit << sh;
        mask |= 255u << sh;
        need = s_need;
    }
    const bool some = budget > recent;  // else no candidate stays
    const int ties = need;
    // warp w: positions [w0, w1) of the share
    const int per = ((x1 - x0 + EV_WARPS - 1) / EV_WARPS + 31) & ~31;
    const int w0 = min(x1, x0 + warp * per), w1 = min(x1, w0 + per);
    int n_eq = 0, n_gt = 0;  // candidates equal to the threshold; those above it and the recent ones
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int pos = i0 + lane;
        const bool c = pos < cand && pos < w1 && some;
        const uint32_t key = c ? key_of(pos) : 0u;
        n_eq += __popc(__ballot_sync(FULL, c && key == prefix));
        n_gt += __popc(__ballot_sync(FULL, (c && key > prefix) || (pos >= cand && pos < w1)));
    }
    if (lane == 0) s_eq[warp] = n_eq, s_keep[warp] = n_gt;
    __syncthreads();
    if (tid == 0) {
        int e = 0, g = 0;
        for (int w = 0; w < EV_WARPS; ++w) e += s_eq[w], g += s_keep[w];
        s_share[0] = e, s_share[1] = g;
    }
    cluster.sync();
    int eq = 0, at = 0;  // equal candidates, kept positions before this warp's range
    for (int r = 0; r < rank; ++r) {
        const int *o = cluster.map_shared_rank(s_share, r);
        at += o[1] + max(0, min(o[0], ties - eq));
        eq += o[0];
    }
    for (int w = 0; w < warp; ++w) {
        at += s_keep[w] + max(0, min(s_eq[w], ties - eq));
        eq += s_eq[w];
    }
    int first = 0x7fffffff;  // first entry that moves
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int pos = i0 + lane;
        const bool c = pos < cand && pos < w1 && some;
        const uint32_t key = c ? key_of(pos) : 0u;
        const uint32_t be = __ballot_sync(FULL, c && key == prefix), below = (1u << lane) - 1u;
        const bool keep = (c && key > prefix) || (pos >= cand && pos < w1) ||
                          (c && key == prefix && eq + __popc(be & below) < ties);
        const uint32_t bk = __ballot_sync(FULL, keep);
        const int j = at + __popc(bk & below);
        if (keep) {
            list[j] = pos;
            if (j != pos) first = min(first, j);
        }
        eq += __popc(be);
        at += __popc(bk);
    }
    first = __reduce_min_sync(FULL, first);
    if (lane == 0) atomicMin(&s_first, first);
    __threadfence();  // the list is read by the other CTAs
    cluster.sync();
    for (int r = 0; r < CS; ++r) first = min(first, *cluster.map_shared_rank(&s_first, r));
    // move: units of sizeof(U) bytes, `per_row` to a row of K or V, then the weights
    const int per_row = rb / (int)sizeof(U);
    const int units = 2 * per_row;
    const int64_t end = (int64_t)budget * units;
    for (int64_t u0 = (int64_t)min(first, budget) * units; u0 < end; u0 += (int64_t)CS * EV_THREADS * EV_UNITS) {
        U v[EV_UNITS];
        U *to[EV_UNITS];
#pragma unroll
        for (int k = 0; k < EV_UNITS; ++k) {
            const int64_t u = u0 + ((int64_t)k * CS + rank) * EV_THREADS + tid;
            to[k] = nullptr;
            if (u < end) {
                const int j = (int)(u / units), part = (int)(u - (int64_t)j * units);
                const int pos = __ldcg(list + j);
                if (pos != j) {
                    uint8_t *base = part < per_row ? kq : vq;
                    const int o = part < per_row ? part : part - per_row;
                    v[k] = *(reinterpret_cast<const U *>(base + row_of(pos) * rb) + o);
                    to[k] = reinterpret_cast<U *>(base + row_of(j) * rb) + o;
                }
            }
        }
        cluster.sync();
#pragma unroll
        for (int k = 0; k < EV_UNITS; ++k)
            if (to[k] != nullptr) *to[k] = v[k];
    }
    for (int j0 = min(first, budget); j0 < budget; j0 += CS * EV_THREADS) {
        const int j = j0 + rank * EV_THREADS + tid;
        const int pos = j < budget ? __ldcg(list + j) : 0;
        const bool moves = j < budget && pos != j;
        const float w = moves ? __ldcg(weights + row_of(pos)) : 0.f;
        cluster.sync();
        if (moves) weights[row_of(j)] = w;
    }
    cluster.sync();  // the others may still be reading this CTA's shared memory
}

cudaError_t launch_paged_evict(const PagedEvictArgs &a)
{
    const Paged p{nullptr, a.lens, a.table, a.B, a.max_pages, a.shift, a.n_pages, 0, 0, a.max_len, a.err};
    const int rb = a.D * a.bits / 8;
    // A CTA to an SM at least, as long as a share has a thousand positions.  Many pairs get small CTAs, whose phases
    // interleave on an SM (512 pairs of 2000 positions cut to 1024, with the read-back: 128 threads 152 us, 256 125,
    // 512 134, 1024 160)
    int cs = 1;
    while (cs < EV_MAX_CLUSTER && (int64_t)a.B * a.H * cs < a.num_sms && a.max_len / (2 * cs) >= 1024) cs *= 2;
    const int cached = std::min(EV_KEYS, (a.max_len / cs + 64) & ~31);
    const bool many = (int64_t)a.B * a.H >= 2 * a.num_sms;
    const void *k16 = many ? (const void *)kv_paged_evict_kernel<uint4, EV_SMALL> : (const void *)kv_paged_evict_kernel<uint4, 1024>;
    const void *k4 = many ? (const void *)kv_paged_evict_kernel<uint32_t, EV_SMALL> : (const void *)kv_paged_evict_kernel<uint32_t, 1024>;
    const void *kern = rb % 16 == 0 ? k16 : k4;
    const size_t smem = (size_t)cached * 4;
    cudaError_t e = kernel_smem(kern, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.B * a.H * cs));
    cfg.blockDim = dim3(many ? EV_SMALL : 1024);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cs;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    void *args[] = {(void *)&a.kq, (void *)&a.vq, (void *)&a.weights, (void *)&p, (void *)&a.H, (void *)&rb, (void *)&a.budget,
                    (void *)&a.recent, (void *)&cached, (void *)&a.new_lens, (void *)&a.kept};
    return cudaLaunchKernelExC(&cfg, kern, args);
}

}  // namespace rptq
