// Blockwise 8-bit copies of bf16 activations: the code of 64 consecutive
// values of a row and their fp32 scale, shared by the kernels that write and
// read such copies (act8.cu, rmsnorm.cu, skinny.cu).
//
// With c the largest magnitude of the block and TOP the code's largest value
// (127 for the linear int8 code, 448 for E4M3),
//   s = fp32(c / TOP),   code = round(TOP x / c),   x~ = bf16_rne(fp32(code s)).
// x and c are bf16, so TOP x has at most 15 significant bits and the exact
// quotient is either a rounding boundary of the code itself or at least
// 2^-17 of its size away from one.  Rounding an fp32 quotient that is off by
// less, and exact at the boundaries, therefore equals rounding the exact one,
// ties included: the codes do not depend on how the division is carried out.
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

// Largest magnitude of the 64 values that kLanes neighbouring lanes hold (8
// with 8 bf16 each, or 4 with 16), as bf16 bits in both
// halves of the result.  As integers the magnitudes order infinities and then
// NaNs above every finite value.
__device__ __forceinline__ uint32_t act8_absmax(const uint4& v) {
    return __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
}
template <int kLanes>
__device__ __forceinline__ uint32_t act8_block_max(uint32_t m) {
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return __vmaxu2(m, prmt(m, m, 0x1032u));
}

// Two fp32 values in one register pair: sm_100 multiplies and adds them in one
// instruction, which halves the arithmetic of the codes.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f2_get(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// What the codes of a block take from its largest magnitude c, and its scale.
// Blocks with c outside [2^-64, 2^64) are first scaled by a power of two so
// that no step leaves the normal range; a value small enough to lose bits
// there has the code 0.
struct Act8Block {
    F2 top, r, neg;        // TOP m, 1 / (c m), -(c m)
    uint32_t keep;         // ~0, or 0 where all codes are 0 (zeros, NaN, infinities)
    float s;
};
template <int kCode>
__device__ __forceinline__ Act8Block act8_block(uint32_t block_max) {
    constexpr float kTop = act8_top<kCode>(), kInvTop = 1.0f / kTop;
    const float c = __uint_as_float(block_max << 16);
    const bool finite = (block_max & 0xffffu) < 0x7f80u;
    Act8Block b;
    // fp32(c / TOP) by Markstein's theorem, from the correctly rounded 1 / TOP,
    // where neither the quotient nor the residual leaves the normal range
    if (c >= 0x1p-90f) {
        const float q0 = __fmul_rn(c, kInvTop);
        b.s = __fmaf_rn(__fmaf_rn(-q0, kTop, c), kInvTop, q0);
    } else {
        b.s = __fdiv_rn(c, kTop);
    }
    if (!finite) b.s = __uint_as_float(0x7fc00000u);
    const float m = c >= 0x1p64f ? 0x1p-64f : c < 0x1p-64f ? 0x1p64f : 1.0f;
    const float cm = __fmul_rn(c, m);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(cm));
    b.top = f2(kTop * m, kTop * m);
    b.r = f2(r, r);
    b.neg = f2(-cm, -cm);
    b.keep = finite && c != 0.f ? 0xffffffffu : 0u;
    return b;
}

// The codes of 8 values of the block.  Per value: a = TOP x (exact), q0 =
// a / c with an approximate 1 / c, the residual a - q0 c (exact as a
// fused multiply-add: 15, 24 and 8 bits, cancelling down to a few units), and
// q0 + residual / c, which is off the exact quotient by 2^-43 of it before its
// rounding: a rounding boundary of the code, an fp32 number, comes out exactly,
// and everything else is 2^-17 away from one.
template <int kCode>
__device__ __forceinline__ uint2 act8_codes(const uint4& v, const Act8Block& b) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    F2 q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const F2 a = f2_mul(f2(bf16lo(w[k]), bf16hi(w[k])), b.top);
        const F2 q0 = f2_mul(a, b.r);
        q[k] = f2_fma(f2_fma(q0, b.neg, a), b.r, q0);
    }
    uint2 c;
    if constexpr (kCode == QLORA_ACT8_E4M3) {
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = __nv_cvt_float2_to_fp8x2(f2_get(q[k]), __NV_SATFINITE, __NV_E4M3);
        c = make_uint2(prmt(h[0], h[1], 0x5410u), prmt(h[2], h[3], 0x5410u));
    } else {
        // |q| <= 127: adding 1.5 2^23 rounds to the nearest integer (ties to
        // even) and leaves its two's complement in the low bits
        const F2 magic = f2(12582912.0f, 12582912.0f);
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 t = f2_get(f2_add(q[k], magic));
            h[k] = prmt(__float_as_uint(t.x), __float_as_uint(t.y), 0x0040u);
        }
        c = make_uint2(prmt(h[0], h[1], 0x5410u), prmt(h[2], h[3], 0x5410u));
    }
    return make_uint2(c.x & b.keep, c.y & b.keep);
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
