// kv_paged_attn.cuh -- what the paged attention kernels share.
//
// Packed codes go to the tensor cores without a conversion.  A code moved to bit position `pos` of an
// otherwise zero 16-bit word is, read as fp16, exactly code * 2^(pos - 24): bits 0-9 are a subnormal's
// mantissa, and bit 10 (exponent field 1, the same spacing of 2^-24) continues it, so 11 bits are linear
// and one mask leaves a code, or one code in each half of a 32-bit word, as a matrix operand.  The power
// of two is taken out of the other operand (queries) or of the result (outputs).
//     x_p = scale sum_d q_d s_d (code_pd - z_d):  the z part is the same for every position of a row and
//           drops out of the softmax;  q'_d = q_d s_d goes in as fp16, scaled by a power of two per row
//           that puts its largest |q'| in [2^14, 2^15);
//     out_d = s_d (sum_p w_p code_pd / sum_p w_p - z_d).
// Where the result must be good to fp32 (fp32 queries; running sums of weights, which are fp32 and
// long-lived) an operand is split into two fp16 parts, 22 bits together; elsewhere q' and w carry fp16's
// 11 bits (an error of 2^-11 at most, below the output's own rounding to bf16 or fp16).
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
    float mid;  // what the codes of V have had taken off in `part`
};

// few rows to a K/V head (kv_paged_decode.cu)
bool paged_decode_takes(int Hq, int H, int D, int dtype, int max_q, int weights);
size_t paged_decode_workspace(int64_t T, int Hq, int H, int D, int dtype, int B, int max_q, int max_len, int weights,
                              int num_sms);
cudaError_t launch_paged_decode(const PagedAttnArgs &a);

}  // namespace rptq
