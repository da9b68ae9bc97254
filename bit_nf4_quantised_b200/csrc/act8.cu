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
// All four kernels are streams: a lane takes 8 values (one 16-byte word of
// bf16, 8 bytes of codes), 8 lanes a block of 64, so the block's maximum is
// three shuffles and every access is a full line of a warp.
#include "act8.cuh"

namespace qnf4 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

template <int kCode>
__global__ void __launch_bounds__(kThreads)
act8_quantize_kernel(const uint4* __restrict__ X, uint2* __restrict__ codes, float* __restrict__ scales,
                     int64_t n8) {
    // n8 is a multiple of 8, so the 8 lanes of a block leave together; the
    // other lanes of the last warp still take part in the shuffles
    for (int64_t i0 = blockIdx.x * int64_t(kThreads); i0 < n8; i0 += int64_t(gridDim.x) * kThreads) {
        const int64_t i = i0 + threadIdx.x;
        const bool live = i < n8;
        const uint4 v = live ? __ldcs(X + i) : make_uint4(0u, 0u, 0u, 0u);
        float s;
        const uint2 c = act8_encode<kCode>(v, act8_absmax(v), &s);
        if (!live) continue;
        codes[i] = c;
        if ((i & 7) == 0) scales[i >> 3] = s;
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
swiglu_forward_act8_kernel(const uint4* __restrict__ G, const uint4* __restrict__ U, uint4* __restrict__ H,
                           uint2* __restrict__ g8, float* __restrict__ gs, uint2* __restrict__ u8,
                           float* __restrict__ us, int64_t n8) {
    for (int64_t i0 = blockIdx.x * int64_t(kThreads); i0 < n8; i0 += int64_t(gridDim.x) * kThreads) {
        const int64_t i = i0 + threadIdx.x;
        const bool live = i < n8;
        const uint4 g = live ? __ldcs(G + i) : make_uint4(0u, 0u, 0u, 0u);
        const uint4 u = live ? __ldcs(U + i) : make_uint4(0u, 0u, 0u, 0u);
        float sg, su;
        const uint2 cg = act8_encode<kCode>(g, act8_absmax(g), &sg);
        const uint2 cu = act8_encode<kCode>(u, act8_absmax(u), &su);
        if (!live) continue;
        const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float g0 = bf16lo(gw[k]), g1 = bf16hi(gw[k]);
            h[k] = pack_bf16x2(g0 * sigmoid(g0) * bf16lo(uw[k]), g1 * sigmoid(g1) * bf16hi(uw[k]));
        }
        __stcs(H + i, make_uint4(h[0], h[1], h[2], h[3]));
        __stcs(g8 + i, cg);
        __stcs(u8 + i, cu);
        if ((i & 7) == 0) {
            gs[i >> 3] = sg;
            us[i >> 3] = su;
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
    const unsigned grid = grid_for(n / 8, num_sms);
    const auto* x = reinterpret_cast<const uint4*>(X);
    auto* c = reinterpret_cast<uint2*>(o.codes);
    if (o.code == QLORA_ACT8_E4M3)
        act8_quantize_kernel<QLORA_ACT8_E4M3><<<grid, kThreads, 0, s>>>(x, c, o.scales, n / 8);
    else
        act8_quantize_kernel<QLORA_ACT8_INT8><<<grid, kThreads, 0, s>>>(x, c, o.scales, n / 8);
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
    const unsigned grid = grid_for(n / 8, num_sms);
    const auto *pg = reinterpret_cast<const uint4*>(G), *pu = reinterpret_cast<const uint4*>(U);
    auto* h = reinterpret_cast<uint4*>(H);
    auto *cg = reinterpret_cast<uint2*>(g.codes), *cu = reinterpret_cast<uint2*>(u.codes);
    if (g.code == QLORA_ACT8_E4M3)
        swiglu_forward_act8_kernel<QLORA_ACT8_E4M3><<<grid, kThreads, 0, s>>>(pg, pu, h, cg, g.scales, cu, u.scales, n / 8);
    else
        swiglu_forward_act8_kernel<QLORA_ACT8_INT8><<<grid, kThreads, 0, s>>>(pg, pu, h, cg, g.scales, cu, u.scales, n / 8);
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
