// kv_paged_attn.cuh -- what the paged attention kernels share.
//
// Packed codes go to the tensor cores without a conversion.  A code moved to bit position `pos` of an
// otherwise zero 16-bit word is, read as fp16, exactly code * 2^(pos - 24): bits 0-9 are a subnormal's
// mantissa, and bit 10 (exponent field 1, the same spacing of 2^-24) continues it, so 11 bits are linear
// and one mask leaves a code, or one code in each half of a 32-bit word, as a matrix operand.  The power
// of two is taken out of the other operand (queries) or of the result (outputs).
//     x_p = scale sum_d q_d s_d (code_pd - z_d):  the z part is the same for every position of a row and
//           drops out of the softmax;  q'_d = q_d s_d goes in scaled by a power of two per row;
//     out_d = s_d (sum_p w_p (code_pd - c_d) / sum_p w_p - (z_d - c_d)),  c_d = 0, or the code nearest to z_d.
// Where more than fp16's 11 bits of an operand are needed (fp32 outputs; the scores behind running sums, which are fp32
// and long-lived) it goes in as several fp16 parts; how many, and on which grid, each kernel says for itself.
#pragma once

#include "kv_paged.cuh"
#include "launch.h"

namespace rptq {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float TWO24 = 16777216.f;

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// element i of a tensor of run-time type
__device__ __forceinline__ float load_elem(const void *p, int dtype, int64_t i)
{
    if (dtype == RPTQ_F32) return static_cast<const float *>(p)[i];
    if (dtype == RPTQ_F16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void store_elem(void *p, int dtype, int64_t i, float v)
{
    if (dtype == RPTQ_F32)
        static_cast<float *>(p)[i] = v;
    else if (dtype == RPTQ_F16)
        static_cast<__half *>(p)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// v as the sum of two fp16 values
__device__ __forceinline__ float fp16_rest(float v) { return v - __half2float(__float2half_rn(v)); }

// cluster id of channel c, checked
__device__ __forceinline__ int cluster_of(const int32_t *cl, int c, int g, int *err)
{
    const int k = cl[c];
    if (k >= 0 && k < g) return k;
    raise_error(err, RPTQ_DEVERR_CLUSTER_ID);
    return 0;
}

// two codes (fp16 subnormals) times 2^14: exact, and normal numbers
__device__ __forceinline__ uint32_t code_up(uint32_t v)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x74007400u));
    return r;
}
// v 2^14 + c
__device__ __forceinline__ uint32_t code_up_plus(uint32_t v, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0x74007400u), "r"(c));
    return r;
}
// The code nearest to a channel's zero point: V's codes enter the precise products less this one, so that a value's error
// is relative to the value (zero stays exactly zero) and not to the step times the code.
__device__ __forceinline__ int zero_code(int z, int qmax) { return min(max(z, 0), qmax); }
// -c 2^(pos - 10), as code_up_plus takes it, for a code c
__device__ __forceinline__ float code_offset(int c, int pos) { return -(float)c * __uint_as_float((uint32_t)(117 + pos) << 23); }
__device__ __forceinline__ uint32_t lds32(const uint8_t *p) { return *reinterpret_cast<const uint32_t *>(p); }

// ---- K: one thread's D / 4 consecutive codes of a row as D / 8 pairs --------------------------------------
// Pair i holds code code(i, 0) at bit pos(i, 0) of the low half and code code(i, 1) at pos(i, 1) of the high
// one.  4-bit: word j gives (8j, 8j+4), (8j+1, 8j+5), ... at positions 0, 4, 0, 4.  3-bit: a 32-bit window whose
// first code is c holds codes c, c+1, c+2 at bits 0, 3, 6 and c+6, c+7, c+8 at 18, 21, 24; two windows three codes
// apart cover 12 codes; the last 8 (D = 128) or 4 (D = 64) are laid into the halves first.
template <int BITS, int D>
struct KPairs {
    static constexpr int N = D / 8;
    __host__ __device__ static constexpr int code(int i, int half)
    {
        if (BITS == 4) return 8 * (i / 4) + i % 4 + 4 * half;
        if (i < (D == 128 ? 12 : 6)) return 12 * (i / 6) + 3 * (i % 6 / 3) + i % 3 + 6 * half;
        return D == 128 ? 24 + (i - 12) + 4 * half : 12 + (i - 6) + 2 * half;
    }
    __host__ __device__ static constexpr int pos(int i, int half)
    {
        if (BITS == 4) return 4 * (i & 1);
        if (i < (D == 128 ? 12 : 6)) return 3 * (i % 3) + 2 * half;
        return D == 128 ? (i == 15 ? 0 : 3 * (i - 12)) : 3 * (i - 6);
    }
    static constexpr int NW = (D / 4 * BITS + 31) / 32;  // words of a quarter
    // the packed words of quarter t of the row at `a` (shared or global memory)
    __device__ __forceinline__ static void read(const uint8_t *a, int t, uint32_t (&w)[NW])
    {
        if constexpr (BITS == 4 && D == 128) {
            const uint4 v = *reinterpret_cast<const uint4 *>(a + 16 * t);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (BITS == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(a + 8 * t);
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (D == 128) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(a + 12 * t);
            w[0] = p[0], w[1] = p[1], w[2] = p[2];
        } else {  // 48 bits at byte 6t
            const uint32_t *p = reinterpret_cast<const uint32_t *>(a + ((6 * t) & ~3));
            const uint32_t wa = p[0], wb = p[1], s = 16 * (t & 1);
            w[0] = __funnelshift_r(wa, wb, s);
            w[1] = wb >> s;
        }
    }
    __device__ __forceinline__ static void expand(const uint32_t (&w)[NW], uint32_t (&x)[N])
    {
        if constexpr (BITS == 4) {
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const uint32_t u = w[j] >> 8;
                x[4 * j] = w[j] & 0x000F000Fu;
                x[4 * j + 1] = w[j] & 0x00F000F0u;
                x[4 * j + 2] = u & 0x000F000Fu;
                x[4 * j + 3] = u & 0x00F000F0u;
            }
        } else if constexpr (D == 128) {
            window(w[0], &x[0]);
            window(__funnelshift_r(w[0], w[1], 9), &x[3]);
            window(__funnelshift_r(w[1], w[2], 4), &x[6]);
            window(__funnelshift_r(w[1], w[2], 13), &x[9]);
            const uint32_t v = w[2] >> 8;  // codes 24..31
            const uint32_t u = (v & 0xFFFu) | ((v << 4) & 0xFFFFF000u);
            x[12] = u & 0x00070007u;
            x[13] = u & 0x00380038u;
            x[14] = u & 0x01C001C0u;
            x[15] = (u >> 9) & 0x00070007u;
        } else {
            window(w[0], &x[0]);
            window(__funnelshift_r(w[0], w[1], 9), &x[3]);
            const uint32_t v = w[1] >> 4;  // codes 12..15
            const uint32_t u = (v & 0x3Fu) | ((v << 10) & 0xFFFF0000u);
            x[6] = u & 0x00070007u;
            x[7] = u & 0x00380038u;
        }
    }
    __device__ __forceinline__ static void load(const uint8_t *a, int t, uint32_t (&x)[N])
    {
        uint32_t w[NW];
        read(a, t, w);
        expand(w, x);
    }
    __device__ __forceinline__ static void window(uint32_t w, uint32_t *x)
    {
        x[0] = w & 0x001C0007u;
        x[1] = w & 0x00E00038u;
        x[2] = w & 0x070001C0u;
    }
};

// Arguments of the kernels for D = 64 and 128.
struct PagedAttnDev {
    Paged p;
    const void *q;
    void *out;
    int dtype, Hq, H, G;
    int64_t q_stride;
    const uint8_t *kq, *vq;
    KvTables kt;
    float scale;
    float *weights;
    // partial results of `splits` parts of the positions: unnormalised sums [splits, T Hq, D], (maximum,
    // sum) [splits, T Hq, 2], and (with weights) the scores [T Hq, max_len], all base 2
    int splits;
    float *part, *ml, *scores;
    float *stat;  // [T Hq, 2] maximum and reciprocal of the sum of each row, for the running sums of a chunk
    int centred;  // V's codes in `part` have had zero_code() taken off (their largest code; 0: nothing)
};

// few rows to a K/V head (kv_paged_decode.cu)
bool paged_decode_takes(int Hq, int H, int D, int dtype, int max_q, int weights);
size_t paged_decode_workspace(int64_t T, int Hq, int H, int D, int dtype, int B, int max_q, int max_len, int weights,
                              int num_sms);
cudaError_t launch_paged_decode(const PagedAttnArgs &a);
// joins the partial results of d.splits parts of the positions
cudaError_t launch_paged_combine(const PagedAttnDev &d, int D, cudaStream_t stream);

// many rows to a K/V head (kv_paged_chunk.cu)
size_t paged_chunk_workspace(int64_t T, int Hq, int H, int D, int dtype, int B, int max_len, int weights, int num_sms);
cudaError_t launch_paged_chunk(const PagedAttnArgs &a);

}  // namespace rptq
