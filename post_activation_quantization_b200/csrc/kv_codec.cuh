// kv_codec.cuh -- the K/V quantizer's arithmetic on a thread's consecutive channels (shared by the
// kernels that quantize whole caches, appended tokens and tokens of a paged cache).
#pragma once

#include "common.cuh"

namespace rptq {

// Correctly rounded x / s from r = RN(1/s): q0 = RN(x r), the residual x - q0 s is exact in
// one fused multiply-add, and q0 + residual * r rounds to RN(x / s) (P. Markstein, "IA-64 and
// Elementary Functions", 2000, division by a reciprocal with one correction).  Quotients that
// are exact half-integers therefore stay exact and round half-to-even like the reference.  The
// residual is exact as long as it is not subnormal: for |x| >= 2^-100 the quotient of every
// finite bf16 or fp16 x is the IEEE one (checked exhaustively by the tests); below, the code is
// decided by rint of a quotient far below 1/2 and does not depend on its last bit.
// The quantizer forms x / (s 2^24) with s' = s 2^24 and r' = RN(1/s) 2^-24 (powers of two: the
// same significands), so that x r' stays finite for every finite x when s >= 2^-24 (no
// inf - inf in the correction), and scales back by 2^24 inside the rounding fma.
__device__ __forceinline__ f32x2 div_rn2(f32x2 x2, f32x2 ns2, f32x2 r2)
{
    const f32x2 q0 = mul2(x2, r2);
    return fma2(fma2(q0, ns2, x2), r2, q0);
}

constexpr int KV_ROWS_PER_UNIT = 64;
constexpr float KV_QSCALE = 16777216.0f;            // 2^24
constexpr float KV_QSCALE_INV = 5.9604644775390625e-08f;  // 2^-24

// Scales s for which the scaled quotient above is exact (no overflow of x r', no overflow or
// subnormal r'); other clusters take the IEEE division.
__device__ __forceinline__ bool kv_fast_scale(float s) { return s >= 0x1p-24f && s <= 0x1p+102f; }

// Coefficients of a thread's DPT channels (h*D + d0 + i) for one head.
template <int BITS, int DPT>
struct KvCoef {
    static constexpr int NG = DPT / 8;
    static constexpr int QMAX = (1 << BITS) - 1;
    static constexpr uint32_t MAGIC_BITS = 0x4B400000u;
    f32x2 ns2[DPT / 2], r2[DPT / 2];  // -s 2^24 and RN(1/s) 2^-24, two channels per pair
    int32_t lo_[DPT], hi_[DPT];       // clamp of the rounded bit pattern: MAGIC_BITS - z .. + qmax
    uint32_t bias[NG];                // sum_i (MAGIC_BITS - z_i) << (BITS*i): removes the rounding constant
    bool fast;                        // every channel: |z| < 2^21 (q + 1.5*2^23 inside one binade) and a fast scale

    __device__ __forceinline__ void load(const int32_t *cl, const float *sc, const int32_t *zp, int c0, int g,
                                         int *err)
    {
        fast = true;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) bias[gi] = 0;
#pragma unroll
        for (int i = 0; i < DPT; i += 2) {
            float sv2[2], rv2[2];
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
                int kc = cl[c0 + i + h2];
                if (kc < 0 || kc >= g) {
                    raise_error(err, RPTQ_DEVERR_CLUSTER_ID);
                    kc = 0;
                }
                const float sv = sc[kc];
                sv2[h2] = sv * KV_QSCALE;
                rv2[h2] = __frcp_rn(sv) * KV_QSCALE_INV;
                const int z = zp[kc];
                lo_[i + h2] = (int32_t)(MAGIC_BITS - (uint32_t)z);
                hi_[i + h2] = (int32_t)(MAGIC_BITS + (uint32_t)QMAX - (uint32_t)z);
                bias[(i + h2) / 8] += (MAGIC_BITS - (uint32_t)z) << (BITS * ((i + h2) % 8));
                fast &= (z > -(1 << 21)) && (z < (1 << 21)) && kv_fast_scale(sv);
            }
            ns2[i / 2] = mk2(-sv2[0], -sv2[1]);
            r2[i / 2] = mk2(rv2[0], rv2[1]);
        }
    }
};

// One code from an IEEE quotient, exactly as the definition: clamp(rint(x / s) + z, 0, qmax)
// (the sum in fp64 is exact for every finite quotient, and an infinite one clamps).
template <int QMAX>
__device__ __forceinline__ uint32_t kv_code_ieee(float x, float s, int z)
{
    const double q = (double)rintf(__fdiv_rn(x, s)) + (double)z;
    return (uint32_t)fmin(fmax(q, 0.0), (double)QMAX);
}

// Codes of one row's DPT channels (x in VEC-element 16-byte chunks) -> NG packed 8-code groups.
template <typename T, int BITS, int DPT>
__device__ __forceinline__ void kv_quant_row(const uint4 *xb, const KvCoef<BITS, DPT> &cf, uint32_t *grp)
{
    constexpr int VEC = Elem<T>::VEC;
    constexpr int NG = DPT / 8;
    const f32x2 magic2 = mk2(MAGIC_RINT, MAGIC_RINT), up2 = mk2(KV_QSCALE, KV_QSCALE);
    if (cf.fast) {
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
            uint32_t acc = 0;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const int i = gi * 8 + j;
                // correctly rounded x / (s 2^24) for two channels, then rint(x / s) + 1.5*2^23:
                // the bit pattern is MAGIC_BITS + rint(x / s) while |x / s| < 2^22; beyond, and
                // for an infinite quotient, it falls outside [lo, hi] on the side of its sign,
                // so the integer clamp below is clamp(rint(x/s), -z, qmax - z) + MAGIC_BITS
                const f32x2 x2 = pair_of<T>(xb[i / VEC], (i % VEC) / 2);
                const f32x2 b2 = fma2(div_rn2(x2, cf.ns2[i / 2], cf.r2[i / 2]), up2, magic2);
                const int32_t l0 = min(max((int32_t)__float_as_uint(lo2(b2)), cf.lo_[i]), cf.hi_[i]);
                const int32_t l1 = min(max((int32_t)__float_as_uint(hi2(b2)), cf.lo_[i + 1]), cf.hi_[i + 1]);
                acc += (uint32_t)l0 << (BITS * j);
                acc += (uint32_t)l1 << (BITS * (j + 1));
            }
            grp[gi] = acc - cf.bias[gi];
        }
    } else {  // a huge zero point or an extreme scale: the IEEE division and the definition
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
            uint32_t acc = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = gi * 8 + j;
                // s and z back from the coefficients (exact: a power-of-two scale, an integer)
                const float sv = -((i & 1) ? hi2(cf.ns2[i / 2]) : lo2(cf.ns2[i / 2])) * KV_QSCALE_INV;
                const int z = (int)(KvCoef<BITS, DPT>::MAGIC_BITS - (uint32_t)cf.lo_[i]);
                acc |= kv_code_ieee<KvCoef<BITS, DPT>::QMAX>(Elem<T>::get(xb[i / VEC], i % VEC), sv, z) << (BITS * j);
            }
            grp[gi] = acc;
        }
    }
}

template <int BITS, int DPT>
__device__ __forceinline__ void kv_store_row(uint8_t *o, const uint32_t *grp)
{
    constexpr int NG = DPT / 8;
    if constexpr (BITS == 4) {
        if constexpr (NG == 2)
            *reinterpret_cast<uint2 *>(o) = make_uint2(grp[0], grp[1]);
        else
            *reinterpret_cast<uint32_t *>(o) = grp[0];
    } else {
        if constexpr (NG == 2) {  // 6 bytes at an even offset: three 2-byte stores
            uint16_t *o16 = reinterpret_cast<uint16_t *>(o);
            o16[0] = (uint16_t)grp[0];
            o16[1] = (uint16_t)((grp[0] >> 16) | (grp[1] << 8));
            o16[2] = (uint16_t)(grp[1] >> 8);
        } else {
            o[0] = (uint8_t)grp[0];
            o[1] = (uint8_t)(grp[0] >> 8);
            o[2] = (uint8_t)(grp[0] >> 16);
        }
    }
}

struct KvTensors {
    const void *src[2];
    uint8_t *dst[2];
    const int32_t *cl[2];
    const float *sc[2];
    const int32_t *zp[2];
};

}  // namespace rptq
