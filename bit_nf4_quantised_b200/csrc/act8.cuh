// Blockwise 8-bit copies of bf16 activations: the code of 64 consecutive
// values of a row and their fp32 scale, shared by the kernels that write and
// read such copies (act8.cu, rmsnorm.cu, skinny.cu).
//
// With c the largest magnitude of the block and TOP the code's largest value
// (127 for the linear int8 code, 448 for E4M3),
//   s = fp32(c / TOP),   code = round(TOP x / c),   x~ = bf16_rne(fp32(code s)).
// x and c are bf16, so TOP x has at most 15 significant bits and the exact
// quotient is either a rounding boundary of the code itself or at least
// 2^-17 of its size away from one.  Rounding the correctly rounded fp32
// quotient therefore equals rounding the exact one, ties included: the codes
// do not depend on how the division is carried out.
// A block of zeros has s = 0; a block with a NaN or an infinity has s = NaN
// and codes 0, so every value of it reads back as NaN.
#pragma once

#include "kernels.cuh"

namespace qnf4 {

__device__ __forceinline__ float bf16lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

template <int kCode>
__host__ __device__ constexpr float act8_top() {
    return kCode == QLORA_ACT8_E4M3 ? 448.0f : 127.0f;
}

// Largest magnitude of the 64 values that 8 neighbouring lanes hold, 8 bf16
// each, as bf16 bits in both halves of the result.  As integers the
// magnitudes order infinities and then NaNs above every finite value.
__device__ __forceinline__ uint32_t act8_absmax(const uint4& v) {
    uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                          __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 4));
    return __vmaxu2(m, prmt(m, m, 0x1032u));
}

// The 8 codes of a lane's values, given act8_absmax of their block; *s is the
// block's scale.  Per value: a = TOP x (exact), q = RN(a r) with r = RN(1/c),
// e = a - q c (exact as a fused multiply-add), and RN(q + e r) is the
// correctly rounded a / c (Markstein's theorem).  Blocks with c outside
// [2^-64, 2^64) are first scaled by a power of two so that no step leaves the
// normal range; a value small enough to lose bits there has the code 0.
template <int kCode>
__device__ __forceinline__ uint2 act8_encode(const uint4& v, uint32_t absmax, float* s) {
    const float c = __uint_as_float(absmax << 16);
    const bool finite = (absmax & 0xffffu) < 0x7f80u;
    *s = finite ? __fdiv_rn(c, act8_top<kCode>()) : __uint_as_float(0x7fc00000u);
    if (!finite || c == 0.f) return make_uint2(0u, 0u);
    const float m = c >= 0x1p64f ? 0x1p-64f : c < 0x1p-64f ? 0x1p64f : 1.0f;
    const float cm = __fmul_rn(c, m), r = __frcp_rn(cm), tm = act8_top<kCode>() * m;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float a = __fmul_rn(k & 1 ? bf16hi(w[k >> 1]) : bf16lo(w[k >> 1]), tm);
        const float q0 = __fmul_rn(a, r);
        q[k] = __fmaf_rn(__fmaf_rn(-q0, cm, a), r, q0);
    }
    if constexpr (kCode == QLORA_ACT8_E4M3) {
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            h[k] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * k], q[2 * k + 1]), __NV_SATFINITE, __NV_E4M3);
        return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    } else {
        // |q| <= 127: adding 1.5 2^23 rounds to the nearest integer (ties to
        // even) and leaves its two's complement in the low bits
        uint32_t b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) b[k] = __float_as_uint(__fadd_rn(q[k], 12582912.0f));
        return make_uint2(prmt(prmt(b[0], b[1], 0x0040u), prmt(b[2], b[3], 0x0040u), 0x5410u),
                          prmt(prmt(b[4], b[5], 0x0040u), prmt(b[6], b[7], 0x0040u), 0x5410u));
    }
}

// fp32(code s) of the four codes in w.
template <int kCode>
__device__ __forceinline__ void act8_decode4(uint32_t w, float s, float (&x)[4]) {
    if (kCode == QLORA_ACT8_E4M3) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            // every E4M3 value is an f16 value
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                static_cast<__nv_fp8x2_storage_t>(k ? w >> 16 : w & 0xffffu), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            x[2 * k] = __fmul_rn(f.x, s);
            x[2 * k + 1] = __fmul_rn(f.y, s);
        }
    } else {
        // code + 128 as the low byte of 2^23, taken off exactly in fp32
        const uint32_t u = w ^ 0x80808080u;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[k] = __fmul_rn(__fsub_rn(__uint_as_float(prmt(u, 0x4b000000u, 0x7540u | k)), 8388736.0f), s);
    }
}

// bf16 pairs of x~ for the eight codes of v.
template <int kCode>
__device__ __forceinline__ uint4 act8_decode8(const uint2& v, float s) {
    float lo[4], hi[4];
    act8_decode4<kCode>(v.x, s, lo);
    act8_decode4<kCode>(v.y, s, hi);
    return make_uint4(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]),
                      pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3]));
}

}  // namespace qnf4
