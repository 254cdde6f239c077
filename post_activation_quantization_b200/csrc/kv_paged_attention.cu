// kv_paged_attention.cu -- attention of each sequence's newest tokens over the paged packed cache.
//
// For token row t = start[b] + i of sequence b (n new tokens, length L) and query head a of K/V head
// h = a / (Hq / H), over the visible positions p <= L - n + i:
//     x_p = scale * sum_d q_d K_pd,   w = softmax(x),   out_d = sum_p w_p V_pd,
// K and V being s (code - z) of their channels; with a pool of running sums, weights[p] of K/V head h
// grows by w_p summed over the sequence's rows and the head's group of query heads.
#include <algorithm>

#include "kv_paged_attn.cuh"

namespace rptq {

// ---- general kernels: every head size ----------------------------------------------------------------
// A lane owns D / 32 consecutive channels of a row.
constexpr int GA_THREADS = 128, GA_WARPS = GA_THREADS / 32, GA_CPL = 8;

struct LaneChannels {
    float s[GA_CPL];
    int z[GA_CPL];
    int n, bit0;  // channels of the lane, first bit of its codes in a row
    __device__ __forceinline__ void load(const int32_t *cl, const float *sc, const int32_t *zp, int c0, int n_, int bits,
                                         int lane, int g, int *err)
    {
        n = n_;
        bit0 = lane * n * bits;
#pragma unroll
        for (int i = 0; i < GA_CPL; ++i) {
            s[i] = 0.f;
            z[i] = 0;
            if (i < n) {
                int k = cl[c0 + i];
                if (k < 0 || k >= g) {
                    raise_error(err, RPTQ_DEVERR_CLUSTER_ID);
                    k = 0;
                }
                s[i] = sc[k];
                z[i] = zp[k];
            }
        }
    }
    // value of the lane's channel i in the packed row
    template <int BITS>
    __device__ __forceinline__ float value(const uint8_t *row, int i) const
    {
        const int bit = bit0 + i * BITS, sh = bit & 7;
        uint32_t w = row[bit >> 3];
        if (sh + BITS > 8) w |= (uint32_t)row[(bit >> 3) + 1] << 8;
        return s[i] * (float)((int)((w >> sh) & ((1u << BITS) - 1u)) - z[i]);
    }
};

// One CTA per (row, query head); its warps take the positions in turn, each with its own running
// maximum and sum (base 2), and are joined at the end.
template <typename T, int BITS>
__global__ void __launch_bounds__(GA_THREADS)
    paged_attention_general(const T *__restrict__ q, int64_t q_stride, Paged p, int Hq, int H, int D,
                            const uint8_t *__restrict__ kq, const uint8_t *__restrict__ vq, KvTables kt, float scale,
                            T *__restrict__ out, float *__restrict__ stat)
{
    __shared__ float s_m[GA_WARPS], s_l[GA_WARPS], s_o[GA_WARPS][GA_CPL * 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x / Hq;
    const int a = (int)(blockIdx.x % Hq), h = a / (Hq / H);
    const int b = paged_row_sequence(p, t);
    int s0, n, L;
    if (b < 0 || !paged_sequence(p, b, s0, n, L)) return;
    const int vis = max(0, L - n + (int)(t - s0) + 1);  // visible positions
    const int cpl = D / 32, rb = D * BITS / 8;
    LaneChannels ck, cv;
    ck.load(kt.ck, kt.sk, kt.zk, h * D + lane * cpl, cpl, BITS, lane, kt.g, p.err);
    cv.load(kt.cv, kt.sv, kt.zv, h * D + lane * cpl, cpl, BITS, lane, kt.g, p.err);
    float qv[GA_CPL], o[GA_CPL];
#pragma unroll
    for (int i = 0; i < GA_CPL; ++i) {
        qv[i] = i < cpl ? to_f32<T>(q[t * q_stride + (int64_t)a * D + lane * cpl + i]) * (scale * LOG2E) : 0.f;
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int pos = warp; pos < vis; pos += GA_WARPS) {
        const int page = max(0, paged_page(p, b, pos >> p.shift));
        const int64_t row = paged_row(page, H, h, p.shift) + (pos & ((1 << p.shift) - 1));
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < GA_CPL; ++i)
            if (i < cpl) x = fmaf(qv[i], ck.value<BITS>(kq + row * rb, i), x);
        for (int f = 16; f > 0; f >>= 1) x += __shfl_xor_sync(FULL, x, f);
        const float mn = fmaxf(m, x);
        const float r = exp2f(m - mn), e = exp2f(x - mn);
        m = mn;
        l = l * r + e;
#pragma unroll
        for (int i = 0; i < GA_CPL; ++i)
            if (i < cpl) o[i] = fmaf(e, cv.value<BITS>(vq + row * rb, i), o[i] * r);
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < GA_CPL; ++i)
        if (i < cpl) s_o[warp][lane * cpl + i] = o[i];
    __syncthreads();
    float mt = s_m[0];
    for (int w = 1; w < GA_WARPS; ++w) mt = fmaxf(mt, s_m[w]);
    float lt = 0.f, f[GA_WARPS];
    for (int w = 0; w < GA_WARPS; ++w) {
        f[w] = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - mt);
        lt += s_l[w] * f[w];
    }
    for (int d = threadIdx.x; d < D; d += GA_THREADS) {
        float v = 0.f;
        for (int w = 0; w < GA_WARPS; ++w) v += f[w] == 0.f ? 0.f : s_o[w][d] * f[w];
        out[(t * Hq + a) * D + d] = from_f32<T>(vis > 0 ? v / lt : 0.f);
    }
    // the row's maximum and the reciprocal of its sum, 0 for a row that sees nothing.  (Their one logarithm would be rounded
    // at the size of the maximum, some thousands where the keys' means are large, and lose the sum's low bits.)
    if (stat != nullptr && threadIdx.x == 0) {
        stat[2 * (t * Hq + a)] = vis > 0 ? mt : 0.f;
        stat[2 * (t * Hq + a) + 1] = vis > 0 ? 1.f / lt : 0.f;
    }
}

// One warp per position of a (sequence, K/V head): its weight summed over the rows that see it, in
// the order of the rows.
template <typename T, int BITS>
__global__ void __launch_bounds__(GA_THREADS)
    paged_weights_general(const T *__restrict__ q, int64_t q_stride, Paged p, int Hq, int H, int D,
                          const uint8_t *__restrict__ kq, KvTables kt, float scale, const float *__restrict__ stat,
                          float *__restrict__ weights)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int bh = blockIdx.x % (p.B * H), b = bh / H, h = bh % H, G = Hq / H;
    int s0, n, L;
    if (!paged_sequence(p, b, s0, n, L) || n == 0) return;
    const int pos = blockIdx.x / (p.B * H) * GA_WARPS + warp;
    if (pos >= L) return;
    const int page = paged_page(p, b, pos >> p.shift);
    if (page < 0) return;
    const int cpl = D / 32, rb = D * BITS / 8;
    const int64_t row = paged_row(page, H, h, p.shift) + (pos & ((1 << p.shift) - 1));
    LaneChannels ck;
    ck.load(kt.ck, kt.sk, kt.zk, h * D + lane * cpl, cpl, BITS, lane, kt.g, p.err);
    float kv[GA_CPL];
#pragma unroll
    for (int i = 0; i < GA_CPL; ++i) kv[i] = i < cpl ? ck.value<BITS>(kq + row * rb, i) : 0.f;
    float w = 0.f;
    for (int i = max(0, pos - (L - n)); i < n; ++i)
        for (int j = 0; j < G; ++j) {
            const int64_t t = s0 + i;
            const int a = h * G + j;
            float x = 0.f;
#pragma unroll
            for (int c = 0; c < GA_CPL; ++c)
                if (c < cpl)
                    x = fmaf(to_f32<T>(q[t * q_stride + (int64_t)a * D + lane * cpl + c]) * (scale * LOG2E), kv[c], x);
            for (int f = 16; f > 0; f >>= 1) x += __shfl_xor_sync(FULL, x, f);
            w = fmaf(exp2f(x - stat[2 * (t * Hq + a)]), stat[2 * (t * Hq + a) + 1], w);
        }
    if (lane == 0) weights[row] += w;
}

size_t paged_attention_workspace(int64_t T, int Hq, int H, int D, int dtype, int B, int max_q, int max_len, int weights,
                                 int num_sms)
{
    if (paged_decode_takes(Hq, H, D, dtype, max_q, weights))
        return paged_decode_workspace(T, Hq, H, D, dtype, B, max_q, max_len, weights, num_sms);
    if (D == 64 || D == 128) return paged_chunk_workspace(T, Hq, H, D, dtype, B, max_len, weights, num_sms);
    return weights ? (size_t)T * Hq * 2 * sizeof(float) : 0;
}

template <typename T, int BITS>
static cudaError_t launch_paged_attention_t(const PagedAttnArgs &a)
{
    const Paged p{a.start, a.lens, a.table, a.B, a.max_pages, a.shift, a.n_pages, a.T, a.max_q, a.max_len, a.err};
    const T *q = static_cast<const T *>(a.q);
    const bool sums = a.weights != nullptr && a.max_len > 0;
    float *stat = sums ? static_cast<float *>(a.ws) : nullptr;
    paged_attention_general<T, BITS><<<(unsigned)(a.T * a.Hq), GA_THREADS, 0, a.stream>>>(
        q, a.q_stride, p, a.Hq, a.H, a.D, a.kq, a.vq, a.kt, a.scale, static_cast<T *>(a.out), stat);
    if (sums)
        paged_weights_general<T, BITS>
            <<<(unsigned)((int64_t)((a.max_len + GA_WARPS - 1) / GA_WARPS) * a.B * a.H), GA_THREADS, 0, a.stream>>>(
                q, a.q_stride, p, a.Hq, a.H, a.D, a.kq, a.kt, a.scale, stat, a.weights);
    return cudaGetLastError();
}

cudaError_t launch_paged_attention(const PagedAttnArgs &a)
{
    if (a.max_len > 0) {  // else no position anywhere: rows of zeros, no sums, and a workspace of no bytes
        if (paged_decode_takes(a.Hq, a.H, a.D, a.dtype, a.max_q, a.weights != nullptr)) return launch_paged_decode(a);
        if (a.D == 64 || a.D == 128) return launch_paged_chunk(a);
    }
    switch (a.dtype) {
    case RPTQ_F32: return a.bits == 4 ? launch_paged_attention_t<float, 4>(a) : launch_paged_attention_t<float, 3>(a);
    case RPTQ_F16: return a.bits == 4 ? launch_paged_attention_t<__half, 4>(a) : launch_paged_attention_t<__half, 3>(a);
    default:
        return a.bits == 4 ? launch_paged_attention_t<__nv_bfloat16, 4>(a) : launch_paged_attention_t<__nv_bfloat16, 3>(a);
    }
}

}  // namespace rptq
