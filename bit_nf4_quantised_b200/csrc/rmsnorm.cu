// RMSNorm in front of an adapted layer, with the residual's addition:
//   h = bf16(x + r),  y = bf16(h rstd w),  rstd = 1 / sqrt(mean(h^2) + eps)
// and, in the same pass, y's blockwise 8-bit copy (act8.cuh) for the layer's
// backward.  The norm's weight is fp32 ("QLoRA, explained", "Failure modes",
// "Silent fp32 casts": preparing a model for k-bit training casts its norms
// to fp32).  Backward, with t = w dy:
//   dx = rstd (t - h rstd^2 mean(h t)) + dr,   dw = sum over rows of dy h rstd
// rstd is formed again from h, which the backward reads anyway, in the same
// reduction as mean(h t): nothing but h is kept from the forward.
//
// Both directions are streams bounded by HBM: forward 2 + 2 (+2) bytes read
// and 2 + 2 (+1 1/16) written per element, backward 4 (+2) read, 2 written.
// Each tensor crosses HBM once: a row is spread over the lanes of a warp (up
// to 1024 values) or a CTA, 8 bf16 a lane and 16-byte word, NV words a lane.
// The grid is persistent: a lane keeps its columns of w (and of dw) in
// registers over all its rows, and the next rows arrive by asynchronous copies
// in a ring of shared memory, where each thread reads back only its own words.
// (Held in registers instead, the next row left too few of them: backward
// with residual and dw, 8192 x 4096, 69 us, so 46; 1024 x 16384, 334, so 31.)
// Measured, us, % of a 6568 GB/s copy: 8192 x 4096 forward with residual 47.3
// (86%), with the int8 copy 55.2 (84%); backward with residual and dw 46.4
// (88%), without either 34.7 (88%); 513 x 1088 forward 2.6, backward 6.5;
// 1 x 4096 forward 2.6.  At both ends of the widths dw costs more than its
// traffic, for a cause not found: with residual and dw 1024 x 16384 30.8 (66%; the
// partial rows of dw, written and read, are as much as 160 rows, 3 us of the 10
// above the copy's time) and 16384 x 1024 30.6 (67%; 1.2 MB of them, nothing),
// without dw and residual 17.2 (89%) and 15.1.  Forward 1024 x 16384 20.5.
// Spills, bytes a thread: forward with an 8-bit copy and two words a lane 12
// (with residual 20), backward with residual, dw and one word 12.
#include <algorithm>

#include "act8.cuh"

namespace qnf4 {

namespace {

constexpr int kWarpRowMax = 1024;      // widest row that a single warp takes
constexpr int kWarpRows = 8;           // warps (rows) of such a CTA
constexpr int kMaxWidth = 16384;       // 512 lanes x 4 words x 8 values

// Threads of the largest CTA that holds NV words of a row per lane.
__host__ __device__ constexpr int max_threads(int nv) { return nv == 1 ? 1024 : 512; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the row's warps, in warp order; buf holds one float per warp and
// alternates between two buffers, so one barrier per row is enough.
__device__ __forceinline__ float row_sum(float v, float* buf, int nwarps) {
    v = warp_sum(v);
    if (nwarps == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < nwarps; ++i) s += buf[i];
    return s;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows in flight per row of threads in a kernel's ring, and its bytes.
__host__ __device__ constexpr int pick(int nv, int s1, int s2, int s4) { return nv == 1 ? s1 : nv == 2 ? s2 : s4; }
__host__ __device__ constexpr int forward_stages(int nv) { return pick(nv, 3, 2, 2); }
__host__ __device__ constexpr int backward_stages(int nv) { return pick(nv, 4, 3, 2); }
__host__ __device__ constexpr int forward_ring(int nv, bool res, int threads) {
    return forward_stages(nv) * nv * (res ? 2 : 1) * 16 * threads;
}
__host__ __device__ constexpr int backward_ring(int nv, bool res, int threads) {
    return backward_stages(nv) * nv * (res ? 3 : 2) * 16 * threads;
}

template <int NV, bool kRes, int kCode>      // kCode < 0: no 8-bit copy
__global__ void __launch_bounds__(max_threads(NV))
rmsnorm_forward_kernel(RmsNormArgs a) {
    constexpr int S = forward_stages(NV), kTensors = kRes ? 2 : 1;
    __shared__ float red[2][32];
    extern __shared__ __align__(16) uint8_t ring[];
    const int nvec = a.D / 8, lanes = blockDim.x, nwarps = lanes / 32, threads = blockDim.x * blockDim.y;
    const int64_t stride = int64_t(gridDim.x) * blockDim.y;
    int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const float inv_d = 1.0f / static_cast<float>(a.D);

    // The ring: [stage][word k][tensor][thread]; a thread reads back only what
    // it copied itself, so its own wait is all the synchronisation there is.
    uint8_t* const mine = ring + (threadIdx.y * lanes + threadIdx.x) * 16;
    auto slot = [&](int stage, int k, int t) { return mine + ((stage * NV + k) * kTensors + t) * threads * 16; };
    auto load = [&](int64_t m, int stage) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = threadIdx.x + k * lanes;
            const bool in = m < a.M && v < nvec;
            const int64_t at = in ? m * a.D + v * 8 : 0;
            cp_async16(smem_u32(slot(stage, k, 0)), a.X + at, in ? 16 : 0);        // 0: zeros
            if (kRes) cp_async16(smem_u32(slot(stage, k, 1)), a.R + at, in ? 16 : 0);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        if (row + i * stride < a.M) load(row + i * stride, i);
        else cp_async_commit();
    }
    float w[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = threadIdx.x + k * lanes;
        float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
        if (v < nvec) {
            lo = __ldg(reinterpret_cast<const float4*>(a.weight) + 2 * v);
            hi = __ldg(reinterpret_cast<const float4*>(a.weight) + 2 * v + 1);
        }
        w[k][0] = lo.x; w[k][1] = lo.y; w[k][2] = lo.z; w[k][3] = lo.w;
        w[k][4] = hi.x; w[k][5] = hi.y; w[k][6] = hi.z; w[k][7] = hi.w;
    }
    int stage = 0;
    // rows of a CTA leave the loop together, so its barriers stay aligned
    for (int it = 0; row - threadIdx.y < a.M; row += stride, ++it) {
        load(row + (S - 1) * stride, stage == 0 ? S - 1 : stage - 1);
        cp_async_wait<S - 1>();
        uint32_t h[NV][4];
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint4 x = *reinterpret_cast<const uint4*>(slot(stage, k, 0));
            uint4 r = make_uint4(0u, 0u, 0u, 0u);
            if (kRes) r = *reinterpret_cast<const uint4*>(slot(stage, k, 1));
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[k][j] = kRes ? pack_bf16x2(bf16lo(xw[j]) + bf16lo(rw[j]), bf16hi(xw[j]) + bf16hi(rw[j])) : xw[j];
                ss = fmaf(bf16lo(h[k][j]), bf16lo(h[k][j]), ss);
                ss = fmaf(bf16hi(h[k][j]), bf16hi(h[k][j]), ss);
            }
        }
        const bool live = row < a.M;
        if (a.H != nullptr && live) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = threadIdx.x + k * lanes;
                if (v < nvec)
                    __stcs(reinterpret_cast<uint4*>(a.H + row * a.D + v * 8),
                           make_uint4(h[k][0], h[k][1], h[k][2], h[k][3]));
            }
        }
        const float rstd = __frsqrt_rn(fmaf(row_sum(ss, red[it & 1], nwarps), inv_d, a.eps));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = threadIdx.x + k * lanes;
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = pack_bf16x2(bf16lo(h[k][j]) * rstd * w[k][2 * j], bf16hi(h[k][j]) * rstd * w[k][2 * j + 1]);
            const uint4 yv = make_uint4(y[0], y[1], y[2], y[3]);
            const bool mine = live && v < nvec;
            if (a.Y != nullptr && mine) __stcs(reinterpret_cast<uint4*>(a.Y + row * a.D + v * 8), yv);
            if (kCode >= 0) {
                // D is a multiple of 64: a block's 8 lanes are all inside or all outside the row
                constexpr int code = kCode < 0 ? 0 : kCode;
                const Act8Block b = act8_block<code>(act8_block_max<8>(act8_absmax(yv)));
                const uint2 c = act8_codes<code>(yv, b);
                if (mine) {
                    const int64_t i = row * nvec + v;
                    __stcs(reinterpret_cast<uint2*>(a.q.codes) + i, c);
                    if ((v & 7) == 0) a.q.scales[i >> 3] = b.s;
                }
            }
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    cp_async_wait<0>();
}

// A load that the compiler does not replace by the registers of an earlier one.
__device__ __forceinline__ uint4 lds_again(const void* p) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem_u32(p)));
    return v;
}

template <int NV, bool kRes, bool kWeight>
__global__ void __launch_bounds__(max_threads(NV))
rmsnorm_backward_kernel(RmsNormGradArgs a) {
    constexpr int S = backward_stages(NV), kTensors = kRes ? 3 : 2;
    __shared__ float red[2][2][32];
    extern __shared__ __align__(16) uint8_t ring[];
    const int nvec = a.D / 8, lanes = blockDim.x, nwarps = lanes / 32, threads = blockDim.x * blockDim.y;
    const int64_t stride = int64_t(gridDim.x) * blockDim.y;
    int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    launch_dependents();                         // the sum of the partial dw waits for this grid

    // The ring: [stage][word k][tensor][thread]; a thread reads back only what
    // it copied itself, so its own wait is all the synchronisation there is.
    uint8_t* const mine = ring + (threadIdx.y * lanes + threadIdx.x) * 16;
    auto slot = [&](int stage, int k, int t) { return mine + ((stage * NV + k) * kTensors + t) * threads * 16; };
    auto load = [&](int64_t m, int stage) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = threadIdx.x + k * lanes;
            const bool in = m < a.M && v < nvec;
            const int64_t at = in ? m * a.D + v * 8 : 0;
            cp_async16(smem_u32(slot(stage, k, 0)), a.dY + at, in ? 16 : 0);       // 0: zeros
            cp_async16(smem_u32(slot(stage, k, 1)), a.H + at, in ? 16 : 0);
            if (kRes) cp_async16(smem_u32(slot(stage, k, 2)), a.dR + at, in ? 16 : 0);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        if (row + i * stride < a.M) load(row + i * stride, i);
        else cp_async_commit();
    }
    float w[NV][8], dw[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = threadIdx.x + k * lanes;
        float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
        if (v < nvec) {
            lo = __ldg(reinterpret_cast<const float4*>(a.weight) + 2 * v);
            hi = __ldg(reinterpret_cast<const float4*>(a.weight) + 2 * v + 1);
        }
        w[k][0] = lo.x; w[k][1] = lo.y; w[k][2] = lo.z; w[k][3] = lo.w;
        w[k][4] = hi.x; w[k][5] = hi.y; w[k][6] = hi.z; w[k][7] = hi.w;
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = 0.f;
    }
    int stage = 0;
    for (int it = 0; row - threadIdx.y < a.M; row += stride, ++it) {
        load(row + (S - 1) * stride, stage == 0 ? S - 1 : stage - 1);
        cp_async_wait<S - 1>();
        uint4 gc[NV], xc[NV];
        float ss = 0.f, st = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            gc[k] = *reinterpret_cast<const uint4*>(slot(stage, k, 0));
            xc[k] = *reinterpret_cast<const uint4*>(slot(stage, k, 1));
            const uint32_t gw[4] = {gc[k].x, gc[k].y, gc[k].z, gc[k].w}, xw[4] = {xc[k].x, xc[k].y, xc[k].z, xc[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float h0 = bf16lo(xw[j]), h1 = bf16hi(xw[j]);
                ss = fmaf(h0, h0, ss);
                ss = fmaf(h1, h1, ss);
                st = fmaf(bf16lo(gw[j]) * w[k][2 * j], h0, st);
                st = fmaf(bf16hi(gw[j]) * w[k][2 * j + 1], h1, st);
            }
        }
        ss = warp_sum(ss);
        st = warp_sum(st);
        if (nwarps > 1) {
            float(*buf)[32] = red[it & 1];
            if ((threadIdx.x & 31) == 0) {
                buf[0][threadIdx.x >> 5] = ss;
                buf[1][threadIdx.x >> 5] = st;
            }
            __syncthreads();
            ss = st = 0.f;
            for (int i = 0; i < nwarps; ++i) {
                ss += buf[0][i];
                st += buf[1][i];
            }
        }
        const float rstd = __frsqrt_rn(fmaf(ss, inv_d, a.eps));
        const float c = rstd * rstd * (st * inv_d);
        const bool live = row < a.M;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = threadIdx.x + k * lanes;
            if (NV == 4 && kWeight) {            // no registers to keep them in
                gc[k] = lds_again(slot(stage, k, 0));
                xc[k] = lds_again(slot(stage, k, 1));
            }
            const uint32_t gw[4] = {gc[k].x, gc[k].y, gc[k].z, gc[k].w}, xw[4] = {xc[k].x, xc[k].y, xc[k].z, xc[k].w};
            uint4 rc = make_uint4(0u, 0u, 0u, 0u);
            if (kRes) rc = *reinterpret_cast<const uint4*>(slot(stage, k, 2));
            const uint32_t rw[4] = {rc.x, rc.y, rc.z, rc.w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float h0 = bf16lo(xw[j]), h1 = bf16hi(xw[j]), g0 = bf16lo(gw[j]), g1 = bf16hi(gw[j]);
                float d0 = rstd * fmaf(-h0, c, g0 * w[k][2 * j]), d1 = rstd * fmaf(-h1, c, g1 * w[k][2 * j + 1]);
                if (kRes) {
                    d0 += bf16lo(rw[j]);
                    d1 += bf16hi(rw[j]);
                }
                o[j] = pack_bf16x2(d0, d1);
                if (kWeight && live) {
                    dw[k][2 * j] = fmaf(g0, h0 * rstd, dw[k][2 * j]);
                    dw[k][2 * j + 1] = fmaf(g1, h1 * rstd, dw[k][2 * j + 1]);
                }
            }
            if (live && v < nvec)
                __stcs(reinterpret_cast<uint4*>(a.dX + row * a.D + v * 8), make_uint4(o[0], o[1], o[2], o[3]));
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    if (!kWeight) return;
    // one partial row of dw per CTA; the warps of a warp-per-row CTA add
    // theirs in warp order through shared memory
    float* const sdw = reinterpret_cast<float*>(ring);
    if (blockDim.y > 1) {
        __syncthreads();                         // every thread is done with its part of the ring
        if (threadIdx.y > 0) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = threadIdx.x + k * lanes;
                if (v < nvec) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) sdw[(threadIdx.y - 1) * a.D + v * 8 + j] = dw[k][j];
                }
            }
        }
        __syncthreads();
        if (threadIdx.y > 0) return;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = threadIdx.x + k * lanes;
        if (v >= nvec) continue;
        for (int q = 1; q < blockDim.y; ++q) {
#pragma unroll
            for (int j = 0; j < 8; ++j) dw[k][j] += sdw[(q - 1) * a.D + v * 8 + j];
        }
        float4* p = reinterpret_cast<float4*>(a.part + int64_t(blockIdx.x) * a.D) + 2 * v;
        p[0] = make_float4(dw[k][0], dw[k][1], dw[k][2], dw[k][3]);
        p[1] = make_float4(dw[k][4], dw[k][5], dw[k][6], dw[k][7]);
    }
}

// dw = (accumulate ? dw : 0) + the sum of the partial rows.  A CTA takes 32
// columns; its warps add interleaved rows and then, in warp order, one
// another's sums: a fixed order.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32)
rmsnorm_dweight_kernel(const float* __restrict__ part, int parts, int D, float* dweight, int accumulate) {
    __shared__ float s[kSumWarps][32];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (col < D) {
#pragma unroll 8
        for (int p = warp; p < parts; p += kSumWarps) t += part[int64_t(p) * D + col];
    }
    s[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && col < D) {
        for (int q = 1; q < kSumWarps; ++q) t += s[q][lane];
        dweight[col] = accumulate ? dweight[col] + t : t;
    }
}

struct Shape {
    int nv;              // 16-byte words a lane holds of a row
    dim3 block;          // lanes of a row x rows of a CTA
    int64_t rows_ctas;   // CTAs if each took blockDim.y rows once
};

// A warp per row up to kWarpRowMax values (16384 x 1024, us: forward with the
// int8 copy 27.4, with a CTA per row 29.9; backward 15.7 and 16.9, but with dw 30.9
// and 28.4: the rule is the forward's and the frozen norm's, and costs dw 2.5).  Above it a CTA per row, with two words a lane, four where 512
// lanes would not cover the row; in the forward, with fewer rows than SMs, one,
// for the shortest path through a row (1 x 4096 with the int8 copy: 2.7 us, with
// two words 3.0; the backward with dw 4.6, with two 4.3).
Shape shape_for(int64_t M, int D, int num_sms, bool forward) {
    const int nvec = D / 8;
    Shape s;
    if (D <= kWarpRowMax) {
        s.nv = nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4;
        const int64_t per = (M + num_sms - 1) / num_sms;
        s.block = dim3(32, static_cast<unsigned>(per < kWarpRows ? (per < 1 ? 1 : per) : kWarpRows));
    } else {
        s.nv = nvec > 2 * max_threads(2) ? 4 : forward && M <= num_sms && nvec <= max_threads(1) ? 1 : 2;
        s.block = dim3(static_cast<unsigned>((nvec + s.nv * 32 - 1) / (s.nv * 32) * 32), 1);
    }
    s.rows_ctas = (M + s.block.y - 1) / s.block.y;
    return s;
}

// CTAs of the persistent grid: threads resident at the kernels' register use
unsigned grid_for(const Shape& s, int num_sms, int threads_per_sm) {
    const int per_sm = threads_per_sm / static_cast<int>(s.block.x * s.block.y);
    const int64_t cap = int64_t(num_sms) * (per_sm < 1 ? 1 : per_sm);
    return static_cast<unsigned>(s.rows_ctas < cap ? s.rows_ctas : cap);
}

// Threads per SM that a kernel's registers and ring allow, taken over by its
// persistent grid: forward 1024, or 512 where a lane holds four words of a
// CTA's row.  (8192 x 4096 with 768: 49 us and 1024: 47; the backward with
// residual and dw with 512: 46, 768: 55, 1024: 49.)
int forward_threads(const Shape& s) { return s.nv == 4 && s.block.y == 1 ? 512 : 1024; }
constexpr int kBackwardThreads = 512;

constexpr int kSmemDefault = 47 * 1024;   // dynamic shared memory beside the static, without asking for more

// A kernel's limit is a constant, the ring of its largest CTA: set to the size
// of a call, it would be too low for a larger ring that another host thread is
// about to launch.
template <class Kernel>
cudaError_t allow_smem(Kernel* kernel, int smem, int most) {
    if (smem <= kSmemDefault) return cudaSuccess;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

template <int NV, bool kRes>
cudaError_t run_forward(const RmsNormArgs& a, const Shape& s, unsigned grid, cudaStream_t st) {
    const int smem = forward_ring(NV, kRes, static_cast<int>(s.block.x * s.block.y));
    auto* kernel = a.q.codes == nullptr ? rmsnorm_forward_kernel<NV, kRes, -1>
                   : a.q.code == QLORA_ACT8_E4M3 ? rmsnorm_forward_kernel<NV, kRes, QLORA_ACT8_E4M3>
                                                 : rmsnorm_forward_kernel<NV, kRes, QLORA_ACT8_INT8>;
    const cudaError_t e = allow_smem(kernel, smem, forward_ring(NV, kRes, max_threads(NV)));
    if (e != cudaSuccess) return e;
    kernel<<<grid, s.block, smem, st>>>(a);
    return cudaGetLastError();
}

template <int NV>
cudaError_t run_forward(const RmsNormArgs& a, const Shape& s, unsigned grid, cudaStream_t st) {
    return a.R != nullptr ? run_forward<NV, true>(a, s, grid, st) : run_forward<NV, false>(a, s, grid, st);
}

template <int NV, bool kRes>
cudaError_t run_backward(const RmsNormGradArgs& a, const Shape& s, unsigned grid, cudaStream_t st) {
    // the ring; at the end the partial dw of all rows of threads but one
    constexpr int most = backward_ring(NV, kRes, max_threads(NV));
    static_assert(most >= (kWarpRows - 1) * kWarpRowMax * 4, "the largest ring holds the partial dw too");
    const int threads = static_cast<int>(s.block.x * s.block.y);
    const int smem = std::max(backward_ring(NV, kRes, threads), static_cast<int>(s.block.y - 1) * a.D * 4);
    auto* kernel = a.dweight ? rmsnorm_backward_kernel<NV, kRes, true> : rmsnorm_backward_kernel<NV, kRes, false>;
    const cudaError_t e = allow_smem(kernel, smem, most);
    if (e != cudaSuccess) return e;
    kernel<<<grid, s.block, smem, st>>>(a);
    return cudaGetLastError();
}

template <int NV>
cudaError_t run_backward(const RmsNormGradArgs& a, const Shape& s, unsigned grid, cudaStream_t st) {
    return a.dR != nullptr ? run_backward<NV, true>(a, s, grid, st) : run_backward<NV, false>(a, s, grid, st);
}

}  // namespace

int rmsnorm_max_width() { return kMaxWidth; }

int rmsnorm_parts(int64_t M, int D, int num_sms) {
    return static_cast<int>(grid_for(shape_for(M, D, num_sms, false), num_sms, kBackwardThreads));
}

cudaError_t launch_rmsnorm_forward(const RmsNormArgs& a, int num_sms, cudaStream_t st) {
    const Shape s = shape_for(a.M, a.D, num_sms, true);
    const unsigned grid = grid_for(s, num_sms, forward_threads(s));
    return s.nv == 1 ? run_forward<1>(a, s, grid, st)
           : s.nv == 2 ? run_forward<2>(a, s, grid, st) : run_forward<4>(a, s, grid, st);
}

cudaError_t launch_rmsnorm_backward(const RmsNormGradArgs& a, int num_sms, cudaStream_t st) {
    const Shape s = shape_for(a.M, a.D, num_sms, false);
    const unsigned grid = grid_for(s, num_sms, kBackwardThreads);
    const cudaError_t e = s.nv == 1 ? run_backward<1>(a, s, grid, st)
                          : s.nv == 2 ? run_backward<2>(a, s, grid, st) : run_backward<4>(a, s, grid, st);
    if (e != cudaSuccess || a.dweight == nullptr) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.D + 31) / 32));
    cfg.blockDim = dim3(kSumWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rmsnorm_dweight_kernel, static_cast<const float*>(a.part),
                              static_cast<int>(grid), a.D, a.dweight, a.accumulate);
}

}  // namespace qnf4
