// Activation checkpoints in 8 bits: a bf16 activation kept as blockwise 8-bit
// codes with fp32 scales (act8.cuh), read back as bf16, and the SwiGLU whose
// backward reads its two inputs from such copies:
//   forward   h = bf16(silu(g) u), and the 8-bit copies of g and u
//   backward  from g~, u~: dg = bf16(dh u~ silu'(g~)), du = bf16(dh silu(g~)),
//             and, if asked for, h~ = bf16(silu(g~) u~)
// silu(z) = z s, silu'(z) = s (1 + z (1 - s)), s = 1 / (1 + exp(-z)), in fp32.
// Checkpointing ("QLoRA, explained", "The algorithm, step by step"; "Compute
// and memory cost") otherwise keeps only the layer's input and recomputes g
// and u through two dequantising GEMMs.
//
// All four kernels are streams bounded by HBM.  The writers take 16 values a
// lane, so that a block's maximum is two shuffles and its constants (scale,
// reciprocal) are formed by 4 lanes; with 8 values a lane, their arithmetic
// took more time than the traffic (8192 x 11008, int8, us: copy 63 -> 46.8,
// SwiGLU forward 186 -> 143).  The readers take 8, a 16-byte word of bf16.
// Measured at 8192 x 11008, us, % of a 6568 GB/s copy: copy int8 46.8 (90%),
// E4M3 47.0; reading back 48.3 (87%); SwiGLU forward 143 (78%: the division
// of its sigmoid, which has to be the correctly rounded one for h to be the
// h of the path without copies), backward 134 int8 (83%), 130 E4M3 (86%).
#include "act8.cuh"

namespace qnf4 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// 16 values a lane: the block's constants are formed by 4 lanes in place of 8.
template <int kCode>
__global__ void __launch_bounds__(kThreads)
act8_quantize_kernel(const uint4* __restrict__ X, uint4* __restrict__ codes, float* __restrict__ scales,
                     int64_t n16) {
    // n16 is a multiple of 4, so the 4 lanes of a block leave together; the
    // other lanes of the last warp still take part in the shuffles
    for (int64_t i0 = blockIdx.x * int64_t(kThreads); i0 < n16; i0 += int64_t(gridDim.x) * kThreads) {
        const int64_t i = i0 + threadIdx.x;
        uint4 v[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (i < n16) {
            v[0] = __ldcs(X + 2 * i);
            v[1] = __ldcs(X + 2 * i + 1);
        }
        const Act8Block b = act8_block<kCode>(act8_block_max<4>(__vmaxu2(act8_absmax(v[0]), act8_absmax(v[1]))));
        if (i >= n16) continue;
        const uint2 lo = act8_codes<kCode>(v[0], b), hi = act8_codes<kCode>(v[1], b);
        codes[i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        if ((i & 3) == 0) scales[i >> 2] = b.s;
    }
}

template <int kCode>
__global__ void __launch_bounds__(kThreads)
act8_dequantize_kernel(const uint2* __restrict__ codes, const float* __restrict__ scales,
                       uint4* __restrict__ X, int64_t n8) {
    for (int64_t i = blockIdx.x * int64_t(kThreads) + threadIdx.x; i < n8;
         i += int64_t(gridDim.x) * kThreads)
        __stcs(X + i, act8_decode8<kCode>(__ldcs(codes + i), __ldg(scales + (i >> 3))));
}

template <int kCode>
__global__ void __launch_bounds__(kThreads)
swiglu_forward_act8_kernel(const uint4* G, const uint4* U, uint4* H,
                           uint4* __restrict__ g8, float* __restrict__ gs, uint4* __restrict__ u8,
                           float* __restrict__ us, int64_t n16) {
    for (int64_t i0 = blockIdx.x * int64_t(kThreads); i0 < n16; i0 += int64_t(gridDim.x) * kThreads) {
        const int64_t i = i0 + threadIdx.x;
        uint4 g[2], u[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            g[e] = u[e] = make_uint4(0u, 0u, 0u, 0u);
            if (i < n16) {
                g[e] = __ldcs(G + 2 * i + e);
                u[e] = __ldcs(U + 2 * i + e);
            }
        }
        const Act8Block bg = act8_block<kCode>(act8_block_max<4>(__vmaxu2(act8_absmax(g[0]), act8_absmax(g[1]))));
        const Act8Block bu = act8_block<kCode>(act8_block_max<4>(__vmaxu2(act8_absmax(u[0]), act8_absmax(u[1]))));
        if (i >= n16) continue;
        const uint2 g0 = act8_codes<kCode>(g[0], bg), g1 = act8_codes<kCode>(g[1], bg);
        __stcs(g8 + i, make_uint4(g0.x, g0.y, g1.x, g1.y));
        const uint2 u0 = act8_codes<kCode>(u[0], bu), u1 = act8_codes<kCode>(u[1], bu);
        __stcs(u8 + i, make_uint4(u0.x, u0.y, u1.x, u1.y));
        if ((i & 3) == 0) {
            gs[i >> 2] = bg.s;
            us[i >> 2] = bu.s;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t gw[4] = {g[e].x, g[e].y, g[e].z, g[e].w}, uw[4] = {u[e].x, u[e].y, u[e].z, u[e].w};
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float z0 = bf16lo(gw[k]), z1 = bf16hi(gw[k]);
                h[k] = pack_bf16x2(z0 * sigmoid(z0) * bf16lo(uw[k]), z1 * sigmoid(z1) * bf16hi(uw[k]));
            }
            __stcs(H + 2 * i + e, make_uint4(h[0], h[1], h[2], h[3]));
        }
    }
}

// kGrad: write dG and dU from dH.  kHidden: write H.
template <int kCode, bool kGrad, bool kHidden>
__global__ void __launch_bounds__(kThreads)
swiglu_backward_act8_kernel(const uint4* __restrict__ dH, const uint2* __restrict__ g8,
                            const float* __restrict__ gs, const uint2* __restrict__ u8,
                            const float* __restrict__ us, uint4* __restrict__ dG, uint4* __restrict__ dU,
                            uint4* __restrict__ H, int64_t n8) {
    for (int64_t i = blockIdx.x * int64_t(kThreads) + threadIdx.x; i < n8;
         i += int64_t(gridDim.x) * kThreads) {
        const uint4 g = act8_decode8<kCode>(__ldcs(g8 + i), __ldg(gs + (i >> 3)));
        const uint4 u = act8_decode8<kCode>(__ldcs(u8 + i), __ldg(us + (i >> 3)));
        uint4 d = make_uint4(0u, 0u, 0u, 0u);
        if (kGrad) d = __ldcs(dH + i);
        const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
        const uint32_t dw[4] = {d.x, d.y, d.z, d.w};
        uint32_t dg[4], du[4], h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float gg[2] = {bf16lo(gw[k]), bf16hi(gw[k])}, uu[2] = {bf16lo(uw[k]), bf16hi(uw[k])};
            const float dd[2] = {bf16lo(dw[k]), bf16hi(dw[k])};
            float og[2], ou[2], oh[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float s = sigmoid(gg[e]), silu = gg[e] * s;
                og[e] = dd[e] * uu[e] * (s * (1.0f + gg[e] * (1.0f - s)));
                ou[e] = dd[e] * silu;
                oh[e] = silu * uu[e];
            }
            dg[k] = pack_bf16x2(og[0], og[1]);
            du[k] = pack_bf16x2(ou[0], ou[1]);
            h[k] = pack_bf16x2(oh[0], oh[1]);
        }
        if (kGrad) {
            __stcs(dG + i, make_uint4(dg[0], dg[1], dg[2], dg[3]));
            __stcs(dU + i, make_uint4(du[0], du[1], du[2], du[3]));
        }
        if (kHidden) __stcs(H + i, make_uint4(h[0], h[1], h[2], h[3]));
    }
}

unsigned grid_for(int64_t n8, int num_sms) {
    const int64_t g = (n8 + kThreads - 1) / kThreads, cap = int64_t(num_sms) * 8;
    return static_cast<unsigned>(g < cap ? g : cap);
}

template <int kCode>
cudaError_t swiglu_backward(const uint16_t* dH, const Act8View& g, const Act8View& u, uint16_t* dG, uint16_t* dU,
                            uint16_t* H, int64_t n8, unsigned grid, cudaStream_t s) {
    const auto* d = reinterpret_cast<const uint4*>(dH);
    const auto* gc = reinterpret_cast<const uint2*>(g.codes);
    const auto* uc = reinterpret_cast<const uint2*>(u.codes);
    auto *og = reinterpret_cast<uint4*>(dG), *ou = reinterpret_cast<uint4*>(dU), *oh = reinterpret_cast<uint4*>(H);
    if (dG && H)
        swiglu_backward_act8_kernel<kCode, true, true><<<grid, kThreads, 0, s>>>(d, gc, g.scales, uc, u.scales, og, ou, oh, n8);
    else if (dG)
        swiglu_backward_act8_kernel<kCode, true, false><<<grid, kThreads, 0, s>>>(d, gc, g.scales, uc, u.scales, og, ou, oh, n8);
    else
        swiglu_backward_act8_kernel<kCode, false, true><<<grid, kThreads, 0, s>>>(d, gc, g.scales, uc, u.scales, og, ou, oh, n8);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_act8_quantize(const uint16_t* X, const Act8View& o, int64_t n, int num_sms, cudaStream_t s) {
    const unsigned grid = grid_for(n / 16, num_sms);
    const auto* x = reinterpret_cast<const uint4*>(X);
    auto* c = reinterpret_cast<uint4*>(o.codes);
    if (o.code == QLORA_ACT8_E4M3)
        act8_quantize_kernel<QLORA_ACT8_E4M3><<<grid, kThreads, 0, s>>>(x, c, o.scales, n / 16);
    else
        act8_quantize_kernel<QLORA_ACT8_INT8><<<grid, kThreads, 0, s>>>(x, c, o.scales, n / 16);
    return cudaGetLastError();
}

cudaError_t launch_act8_dequantize(const Act8View& v, uint16_t* X, int64_t n, int num_sms, cudaStream_t s) {
    const unsigned grid = grid_for(n / 8, num_sms);
    const auto* c = reinterpret_cast<const uint2*>(v.codes);
    auto* x = reinterpret_cast<uint4*>(X);
    if (v.code == QLORA_ACT8_E4M3)
        act8_dequantize_kernel<QLORA_ACT8_E4M3><<<grid, kThreads, 0, s>>>(c, v.scales, x, n / 8);
    else
        act8_dequantize_kernel<QLORA_ACT8_INT8><<<grid, kThreads, 0, s>>>(c, v.scales, x, n / 8);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_forward_act8(const uint16_t* G, const uint16_t* U, uint16_t* H, const Act8View& g,
                                       const Act8View& u, int64_t n, int num_sms, cudaStream_t s) {
    const unsigned grid = grid_for(n / 16, num_sms);
    const auto *pg = reinterpret_cast<const uint4*>(G), *pu = reinterpret_cast<const uint4*>(U);
    auto* h = reinterpret_cast<uint4*>(H);
    auto *cg = reinterpret_cast<uint4*>(g.codes), *cu = reinterpret_cast<uint4*>(u.codes);
    if (g.code == QLORA_ACT8_E4M3)
        swiglu_forward_act8_kernel<QLORA_ACT8_E4M3><<<grid, kThreads, 0, s>>>(pg, pu, h, cg, g.scales, cu, u.scales, n / 16);
    else
        swiglu_forward_act8_kernel<QLORA_ACT8_INT8><<<grid, kThreads, 0, s>>>(pg, pu, h, cg, g.scales, cu, u.scales, n / 16);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_backward_act8(const uint16_t* dH, const Act8View& g, const Act8View& u, uint16_t* dG,
                                        uint16_t* dU, uint16_t* H, int64_t n, int num_sms, cudaStream_t s) {
    const unsigned grid = grid_for(n / 8, num_sms);
    return g.code == QLORA_ACT8_E4M3
               ? swiglu_backward<QLORA_ACT8_E4M3>(dH, g, u, dG, dU, H, n / 8, grid, s)
               : swiglu_backward<QLORA_ACT8_INT8>(dH, g, u, dG, dU, H, n / 8, grid, s);
}

}  // namespace qnf4
