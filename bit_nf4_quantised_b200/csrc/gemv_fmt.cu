// Matrix-vector products with a 4-bit weight in any stored format: for 1 to
// 16 tokens,
//   Y[m][n] = sum_k x[m][k] q[idx[n][k]] c~[block(n, k)]  (+ the LoRA term)
// with any codebook of up to 16 codes, blocks of 16 to 4096 weights and fp32
// or 8-bit block scales ("QLoRA, explained", "A toy run: how much does NF4
// lose ..."): decoding on the format variants, as gemv.cu does on the NF4
// storage.
//
// The weight enters as the code and its scale, not as a bf16 product: a block
// shares its scale, so the sum of q x over the block is formed first, by
// tensor-core products of f16 codes with f16 activations accumulated in fp32,
// and then multiplied by c~ in fp32.
//   codes        times a factor s (1, 3, 5, 7 or 15, and a power of two)
//                that makes their f16 rounding smallest: FP4 and INT4 are
//                exact, an NF4 code is off by 2^-12 of itself at most, where
//                one bf16 rounding of Y allows 2^-9.
//   activations  times a power of two per token that puts the token's largest
//                value in [2^14, 2^15): their 8 bits are exact in f16 down to
//                2^-28 of the largest; below, off by 2^-40 of it.
// Both factors are taken out of the sums at the end.
//
// A CTA per SM, 16 warps, each on 16 RG rows and a share of the contraction.
//   weights      straight from HBM to registers, 16 bytes (32 weights) per
//                lane and load, the next 256 columns in flight while the
//                current ones are multiplied.  Lane (g, c) holds rows g and
//                g + 8 of a 16-row group, weights 32 c ... 32 c + 31 of a
//                128-wide chunk; MMA j (of 8 per chunk) multiplies every
//                lane's weights 4 j ... 4 j + 3.
//   expansion    a packed byte addresses a pair of f16 codes in a table with
//                a copy per lane (no bank conflicts): one byte permute and
//                one 4-byte shared load per two weights, no arithmetic.
//   scales       the four lanes of a row hold weights of up to G = 4 blocks,
//                which one MMA must not add up.  The MMA has 8 columns, so a
//                token takes G of them: column (token, b) holds x where the
//                lane's block is b and zero elsewhere, and comes out as the
//                sum over block b alone (blocks of 16 take two sets of MMAs).
//                A warp stages its rows' scales, decoded to fp32, in shared
//                memory 256 columns at a time.
//   joining      the warps' partial sums meet in shared memory once per unit
//                of rows and are added in warp order.  Contraction slices,
//                where a CTA's activations would not fit in shared memory,
//                and the LoRA term are joined by gemv_finalize_kernel.
// Bound: HBM; next to it the shared-memory pipe, one wavefront per 64 weights
// for the table.
#include <cuda_fp16.h>

#include <algorithm>

#include "kernels.cuh"

namespace qnf4 {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kLutBytes = 256 * 256;         // 256 byte values, 64 words apart, 32 lanes' copies

// One variant: G blocks (columns) per token in a chunk, SB sets of MMAs
// (blocks of 16), NT tiles of 8 columns, RG 16-row groups per warp.
template <int G, int SB>
struct Layout {
    static constexpr int kGran = G == 1 ? 128 : G == 2 ? 64 : 32 / SB;   // weights per staged scale
    static constexpr int kPerChunk = 128 / kGran;
    static constexpr int kPerStep = 2 * kPerChunk;                       // per row and 256 columns
    static constexpr int kPitch = kPerStep == 2 ? 2 : kPerStep + 2;      // fp32; 8 rows' pairs meet no bank twice
};

struct Plan {
    int x_pitch, stage, red_pitch, red_bufs;
    int off_x, off_stage, off_red, off_misc, total;
};

// Shared memory: code table, activations, staged scales, partial sums, and
// the tokens' largest magnitudes and factors.
__host__ __device__ inline Plan plan_smem(int M, int chunks, int pitch, int rows_per_warp) {
    Plan p;
    p.x_pitch = ((chunks + 1) / 2 * 2) * 256 + 64;        // 64 mod 128: two tokens' loads share no bank
    p.stage = rows_per_warp * pitch * 4;                  // per warp
    p.red_pitch = rows_per_warp + 8;
    p.red_bufs = M <= 4 ? 2 : 1;
    p.off_x = kLutBytes;
    p.off_stage = p.off_x + M * p.x_pitch;
    p.off_red = p.off_stage + kWarps * p.stage;
    p.off_misc = p.off_red + p.red_bufs * kWarps * M * p.red_pitch * 4;
    p.total = p.off_misc + 2 * 16 * 4;
    return p;
}

__device__ __forceinline__ uint4 ldg_weights(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float decode_scale(uint32_t code, int fmt) {
    return fmt == QLORA_SCALES_E4M3 ? e4m3_to_float(static_cast<uint8_t>(code))
           : fmt == QLORA_SCALES_E5M2 ? e5m2_to_float(static_cast<uint8_t>(code))
                                      : static_cast<float>(code);
}

// A row's scales over 256 columns as loaded: codes and two constants, or fp32.
template <int E, bool kF32>
struct RawScales {
    uint32_t w[kF32 ? E : (E + 3) / 4];
    float m0, m1;
    int split;                            // entries before it belong to m0's group

    // f: flat position of the first entry; last: of the last valid one;
    // vec: entries are consecutive and 4-entry aligned
    __device__ __forceinline__ void load(const GemvFmtArgs& a, int64_t f, int64_t last, int gran, bool vec) {
        const int64_t b0 = f >> a.log2_block;
        if (kF32) {
            const float* s = static_cast<const float*>(a.scales);
            if (E >= 4 && vec) {
#pragma unroll
                for (int e = 0; e < E / 4; ++e) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(s + b0) + e);
                    w[4 * e] = v.x; w[4 * e + 1] = v.y; w[4 * e + 2] = v.z; w[4 * e + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    w[e] = __float_as_uint(__ldg(s + (min(f + e * gran, last) >> a.log2_block)));
            }
            return;
        }
        const uint8_t* s = static_cast<const uint8_t*>(a.scales);
        if (E >= 4 && vec) {
#pragma unroll
            for (int e = 0; e < E / 4; ++e) w[e] = __ldg(reinterpret_cast<const uint32_t*>(s + b0) + e);
        } else {
#pragma unroll
            for (int e = 0; e < (E + 3) / 4; ++e) w[e] = 0;
#pragma unroll
            for (int e = 0; e < E; ++e)
                w[e / 4] |= uint32_t(__ldg(s + (min(f + e * gran, last) >> a.log2_block))) << (8 * (e & 3));
        }
        const int64_t be = min(f + (E - 1) * gran, last) >> a.log2_block;
        m0 = __ldg(a.meta + (b0 >> 8));
        m1 = __ldg(a.meta + (be >> 8));
        // first entry of the next group of 256 blocks
        split = E;
#pragma unroll
        for (int e = E - 1; e > 0; --e)
            if ((((f + e * gran) >> a.log2_block) >> 8) != (b0 >> 8)) split = e;
    }

    __device__ __forceinline__ float get(int e, int fmt) const {
        if (kF32) return __uint_as_float(w[e]);
        return __fmul_rn(decode_scale((w[e / 4] >> (8 * (e & 3))) & 0xffu, fmt), e < split ? m0 : m1);
    }
};

template <int G, int SB, int NT, int RG, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
gemv_fmt_kernel(const __grid_constant__ GemvFmtArgs a) {
    using L = Layout<G, SB>;
    constexpr int kRows = 16 * RG;                        // rows of a warp
    constexpr int kTok = G == 1 ? 4 : 2;                  // totals per tile and lane
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    launch_dependents();

    const int64_t K = a.K;
    const int M = a.M;
    const int64_t k_beg = int64_t(blockIdx.y) * a.chunks * 128;
    const int kslab = static_cast<int>(min(K - k_beg, int64_t(a.chunks) * 128));
    const Plan p = plan_smem(M, a.chunks, L::kPitch, kRows);
    uint8_t* const sx = smem + p.off_x;
    float* const stage = reinterpret_cast<float*>(smem + p.off_stage + warp * p.stage);
    uint32_t* const smax = reinterpret_cast<uint32_t*>(smem + p.off_misc);
    float* const sundo = reinterpret_cast<float*>(smem + p.off_misc + 64);

    // rows of this CTA, and this warp's part of a unit: 16 RG rows (the
    // wr-th such group of the unit) x steps m0 ... m1 - 1 of 256 columns
    const int64_t r0 = a.N * blockIdx.x / gridDim.x, r1 = a.N * (blockIdx.x + 1) / gridDim.x;
    const int wk = warp & (a.warps_k - 1), wr = warp / a.warps_k;
    const int unit_rows = kRows * (kWarps / a.warps_k);
    const int units = static_cast<int>((r1 - r0 + unit_rows - 1) / unit_rows);
    const int steps = (kslab + 255) / 256;
    const int m0 = steps * wk / a.warps_k, m1 = steps * (wk + 1) / a.warps_k;

    uint4 buf[2][RG][2];
    RawScales<L::kPerStep, kF32> raw;
    auto load_chunk = [&](int u, int mi, int cc) {
        const int k = mi * 256 + cc * 128 + c * 32;
#pragma unroll
        for (int q = 0; q < 2 * RG; ++q) {
            const int64_t n = r0 + u * unit_rows + wr * kRows + q * 8 + g;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (n < r1 && k < kslab) v = ldg_weights(a.packed + ((n * K + k_beg + k) >> 1));
            buf[cc][q >> 1][q & 1] = v;
        }
    };
    auto load_scales = [&](int u, int mi) {
        const int64_t n = r0 + u * unit_rows + wr * kRows + lane;
        if (lane < kRows && n < r1) {
            const int64_t row = n * K + k_beg;
            raw.load(a, row + mi * 256, row + kslab - L::kGran, L::kGran, a.vec_scales && mi * 256 + 256 <= kslab);
        }
    };
    auto store_scales = [&]() {
        if (lane < kRows) {
#pragma unroll
            for (int e = 0; e < L::kPerStep; e += 2) {
                // blocks of 16: a chunk's even blocks first, then its odd ones
                float v0 = raw.get(e, a.scale_fmt), v1 = raw.get(e + 1, a.scale_fmt);
                const int ch = e / L::kPerChunk * L::kPerChunk, in = e % L::kPerChunk;
                if (SB == 2) {
                    stage[lane * L::kPitch + ch + in / 2] = v0;
                    stage[lane * L::kPitch + ch + 4 + in / 2] = v1;
                } else {
                    *reinterpret_cast<float2*>(stage + lane * L::kPitch + e) = make_float2(v0, v1);
                }
            }
        }
    };
    // the first loads travel while the table and the activations are set up
    if (m0 < m1 && units > 0) {
        load_scales(0, m0);
        load_chunk(0, m0, 0);
        load_chunk(0, m0, 1);
    }

    // code table: byte e of lane l at 256 e + 4 l
    for (int i = tid; i < 256 * 8; i += kThreads) {
        const int e = i >> 3;
        const uint32_t v = a.code[e & 15] | (uint32_t(a.code[e >> 4]) << 16);
        *reinterpret_cast<uint4*>(smem + e * 256 + (i & 7) * 16) = make_uint4(v, v, v, v);
    }
    // activations: each token's largest finite magnitude, then f16 copies
    // scaled by it, 8 columns (one 16-byte word) at a time, in the order the
    // lanes read them: column 32 c + 8 j + i of a chunk at 64 j + 16 c + 2 i;
    // zeros past the slice
    if (tid < 16) smax[tid] = 0;
    __syncthreads();
    const int words = steps * 32;                           // 16-byte words per token
    for (int m = 0; m < M; ++m) {
        uint32_t mx = 0;
        for (int i = tid; i * 8 < kslab; i += kThreads) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.X + m * K + k_beg) + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t lo = w[q] & 0x7fffu, hi = (w[q] >> 16) & 0x7fffu;
                if (lo < 0x7f80u) mx = max(mx, lo);
                if (hi < 0x7f80u) mx = max(mx, hi);
            }
        }
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (lane == 0) atomicMax(smax + m, mx);
    }
    __syncthreads();
    for (int i = tid; i < M * words; i += kThreads) {
        const int m = i / words, w = i % words;
        const int sh = min(126, 14 + 127 - static_cast<int>(smax[m] >> 7));
        const float f = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
        uint4 o = make_uint4(0u, 0u, 0u, 0u);
        if (w * 8 < kslab) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.X + m * K + k_beg) + w);
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
            uint32_t out[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const __half2 h = __floats2half2_rn(__uint_as_float(in[q] << 16) * f,
                                                    __uint_as_float(in[q] & 0xffff0000u) * f);
                out[q] = *reinterpret_cast<const uint32_t*>(&h);
            }
            o = make_uint4(out[0], out[1], out[2], out[3]);
        }
        const int ch = w >> 4, in_ch = w & 15;
        *reinterpret_cast<uint4*>(sx + m * p.x_pitch + ch * 256 + (in_ch & 3) * 64 + (in_ch >> 2) * 16) = o;
        if (w == 0) sundo[m] = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23) * a.code_undo;
    }
    // this CTA's share of T = X A^T: columns s0 ... s1 - 1 of the slice
    if (a.r > 0 && static_cast<int>(blockIdx.x) < a.t_ctas) {
        const int n8 = kslab / 8;
        const int s0 = static_cast<int>(int64_t(n8) * blockIdx.x / a.t_ctas);
        const int s1 = static_cast<int>(int64_t(n8) * (blockIdx.x + 1) / a.t_ctas);
        float* tp = a.Tpart + (int64_t(blockIdx.y) * a.t_ctas + blockIdx.x) * M * a.r;
        for (int j = warp; j < a.r; j += kWarps) {
            for (int mb = 0; mb < M; mb += 4) {
                float t[4] = {0.f, 0.f, 0.f, 0.f};
                for (int s = s0 + lane; s < s1; s += 32) {
                    const uint4 av = __ldg(reinterpret_cast<const uint4*>(a.A + j * K + k_beg) + s);
                    const uint32_t aw[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (mb + q < M) {
                            const uint4 xv = __ldg(reinterpret_cast<const uint4*>(a.X + (mb + q) * K + k_beg) + s);
                            const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                t[q] = fmaf(__uint_as_float(aw[e] << 16), __uint_as_float(xw[e] << 16), t[q]);
                                t[q] = fmaf(__uint_as_float(aw[e] & 0xffff0000u),
                                            __uint_as_float(xw[e] & 0xffff0000u), t[q]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) t[q] += __shfl_xor_sync(0xffffffffu, t[q], o);
                    if (lane == 0 && mb + q < M) tp[(mb + q) * a.r + j] = t[q];
                }
            }
        }
    }
    __syncthreads();

    // this lane's column of each tile: its token's activations where the
    // column's block is the one the lane's weights belong to
    const int my_block = G == 1 ? 0 : G == 2 ? c >> 1 : c;
    uint32_t xoff[NT];
    bool xon[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int col = 8 * t + g, tok = col / G;
        xon[t] = tok < M && col % G == my_block;
        xoff[t] = static_cast<uint32_t>(p.off_x + tok * p.x_pitch + c * 16);
    }
    const uint32_t lane4 = lane * 4;
    auto code_pair = [&](uint32_t w, uint32_t sel) {
        return *reinterpret_cast<const uint32_t*>(smem + prmt(w, lane4, sel));
    };
    float tot[RG][NT][kTok];
#pragma unroll
    for (int q = 0; q < RG; ++q)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < kTok; ++e) tot[q][t][e] = 0.f;

    for (int u = 0; u < units; ++u) {
        for (int mi = m0; mi < m1; ++mi) {
            const bool more = mi + 1 < m1 || u + 1 < units;
            const int nu = mi + 1 < m1 ? u : u + 1, nm = mi + 1 < m1 ? mi + 1 : m0;
            __syncwarp();
            store_scales();
            __syncwarp();
            if (more) load_scales(nu, nm);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                float d[RG][NT][4];
                const uint32_t xch = static_cast<uint32_t>((2 * mi + cc) * 256);
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) {
                    if (jp % (4 / SB) == 0) {
#pragma unroll
                        for (int q = 0; q < RG; ++q)
#pragma unroll
                            for (int t = 0; t < NT; ++t) d[q][t][0] = d[q][t][1] = d[q][t][2] = d[q][t][3] = 0.f;
                    }
                    uint32_t w[RG][2][4];
#pragma unroll
                    for (int q = 0; q < RG; ++q) {
                        const uint4 lo = buf[cc][q][0], hi = buf[cc][q][1];
                        const uint32_t wl = jp == 0 ? lo.x : jp == 1 ? lo.y : jp == 2 ? lo.z : lo.w;
                        const uint32_t wh = jp == 0 ? hi.x : jp == 1 ? hi.y : jp == 2 ? hi.z : hi.w;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            w[q][j][0] = code_pair(wl, 0x5504u | (2 * j) << 4);
                            w[q][j][1] = code_pair(wh, 0x5504u | (2 * j) << 4);
                            w[q][j][2] = code_pair(wl, 0x5504u | (2 * j + 1) << 4);
                            w[q][j][3] = code_pair(wh, 0x5504u | (2 * j + 1) << 4);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (xon[t]) x = *reinterpret_cast<const uint4*>(smem + xoff[t] + xch + jp * 64);
#pragma unroll
                        for (int q = 0; q < RG; ++q) {
                            mma_f16(d[q][t], w[q][0][0], w[q][0][1], w[q][0][2], w[q][0][3], x.x, x.y);
                            mma_f16(d[q][t], w[q][1][0], w[q][1][1], w[q][1][2], w[q][1][3], x.z, x.w);
                        }
                    }
                    if (jp % (4 / SB) == 4 / SB - 1) {
                        // block sums times their scales: the lane's two columns are
                        // two tokens of one block (G = 1) or two blocks of a token
                        const int set = SB == 2 ? jp / 2 : 0;
#pragma unroll
                        for (int q = 0; q < RG; ++q) {
                            const float* sr = stage + (q * 16 + g) * L::kPitch + cc * L::kPerChunk;
                            if (G == 1) {
                                const float s0 = sr[0], s1 = sr[8 * L::kPitch];
#pragma unroll
                                for (int t = 0; t < NT; ++t) {
                                    tot[q][t][0] = fmaf(s0, d[q][t][0], tot[q][t][0]);
                                    tot[q][t][1] = fmaf(s0, d[q][t][1], tot[q][t][1]);
                                    tot[q][t][kTok - 2] = fmaf(s1, d[q][t][2], tot[q][t][kTok - 2]);
                                    tot[q][t][kTok - 1] = fmaf(s1, d[q][t][3], tot[q][t][kTok - 1]);
                                }
                            } else {
                                const int at = set * 4 + (G == 4 ? 2 * (c & 1) : 0);
                                const float2 s0 = *reinterpret_cast<const float2*>(sr + at);
                                const float2 s1 = *reinterpret_cast<const float2*>(sr + 8 * L::kPitch + at);
#pragma unroll
                                for (int t = 0; t < NT; ++t) {
                                    tot[q][t][0] = fmaf(s0.x, d[q][t][0], fmaf(s0.y, d[q][t][1], tot[q][t][0]));
                                    tot[q][t][1] = fmaf(s1.x, d[q][t][2], fmaf(s1.y, d[q][t][3], tot[q][t][1]));
                                }
                            }
                        }
                    }
                }
                if (more) load_chunk(nu, nm, cc);
            }
        }
        // the unit is complete: partial sums [warp][token][row] to shared
        // memory, then one thread per output adds the warps' in order
        float* red = reinterpret_cast<float*>(smem + p.off_red) + (p.red_bufs == 2 ? (u & 1) * kWarps * M * p.red_pitch : 0);
        float* mine = red + warp * M * p.red_pitch;
#pragma unroll
        for (int q = 0; q < RG; ++q)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (G == 1) {
                    const int tok = 8 * t + 2 * c;
                    float* at = mine + tok * p.red_pitch + q * 16 + g;
                    if (tok < M) {
                        at[0] = tot[q][t][0];
                        at[8] = tot[q][t][kTok - 2];
                    }
                    if (tok + 1 < M) {
                        at[p.red_pitch] = tot[q][t][1];
                        at[p.red_pitch + 8] = tot[q][t][kTok - 1];
                    }
                } else {
                    float v0 = tot[q][t][0], v1 = tot[q][t][1];
                    if (G == 4) {                        // the token's other two blocks
                        v0 += __shfl_xor_sync(0xffffffffu, v0, 1);
                        v1 += __shfl_xor_sync(0xffffffffu, v1, 1);
                    }
                    const int tok = G == 2 ? 4 * t + c : 2 * t + (c >> 1);
                    float* at = mine + tok * p.red_pitch + q * 16 + g;
                    if (tok < M && (G == 2 || (c & 1) == 0)) {
                        at[0] = v0;
                        at[8] = v1;
                    }
                }
#pragma unroll
                for (int e = 0; e < kTok; ++e) tot[q][t][e] = 0.f;
            }
        __syncthreads();
        // a different run of warps for each unit (one barrier per unit is
        // enough with two buffers: whoever adds has done so before the next)
        for (int o = (tid + u * 64) & (kThreads - 1); o < unit_rows * M; o += kThreads) {
            const int m = o / unit_rows, row = o % unit_rows;
            const int64_t n = r0 + u * unit_rows + row;
            if (n >= r1) continue;
            const float* src = red + ((row / kRows) * a.warps_k * M + m) * p.red_pitch + row % kRows;
            float s = 0.f;
            for (int q = 0; q < a.warps_k; ++q) s += src[q * M * p.red_pitch];
            s *= sundo[m];
            if (a.part != nullptr) {
                a.part[(int64_t(blockIdx.y) * M + m) * a.N + n] = s;
            } else {
                const __nv_bfloat16 y = __float2bfloat16_rn(s);
                a.Y[m * a.N + n] = *reinterpret_cast<const uint16_t*>(&y);
            }
        }
        if (p.red_bufs == 1) __syncthreads();
    }
}

template <int G, int SB, int NT>
constexpr int row_groups() {
    return NT >= 8 ? 1 : 2;              // 8 tiles x 2 row groups would not fit in registers
}

template <int G, int SB, int NT, bool kF32>
cudaError_t run(const GemvFmtArgs& a, dim3 grid, int smem, cudaStream_t s) {
    constexpr int RG = row_groups<G, SB, NT>();
    auto* kernel = gemv_fmt_kernel<G, SB, NT, RG, kF32>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <int G, int SB, int NT>
cudaError_t run_scales(const GemvFmtArgs& a, dim3 grid, int smem, cudaStream_t s) {
    return a.scale_fmt == QLORA_SCALES_FP32 ? run<G, SB, NT, true>(a, grid, smem, s)
                                            : run<G, SB, NT, false>(a, grid, smem, s);
}

template <int G, int SB>
cudaError_t run_tiles(int nt, const GemvFmtArgs& a, dim3 grid, int smem, cudaStream_t s) {
    if (nt <= 1) return run_scales<G, SB, 1>(a, grid, smem, s);
    if (nt <= 2) return run_scales<G, SB, 2>(a, grid, smem, s);
    if constexpr (G >= 2) {
        if (nt <= 4) return run_scales<G, SB, 4>(a, grid, smem, s);
    }
    if constexpr (G >= 4) {
        return run_scales<G, SB, 8>(a, grid, smem, s);
    }
    return cudaErrorInvalidValue;
}

// Blocks per 128-wide chunk of a row.  Rows of an odd number of 64-wide runs
// shift a block of 128 or more against the next row's chunks by half a chunk,
// so there each run takes its own scale.
void shape_of(int log2_block, int64_t K, int* G, int* SB) {
    *SB = log2_block == 4 ? 2 : 1;
    *G = log2_block <= 5 ? 4 : log2_block == 6 || K % 128 != 0 ? 2 : 1;
}

int pitch_of(int G, int SB) {
    return G == 1 ? Layout<1, 1>::kPitch : G == 2 ? Layout<2, 1>::kPitch
           : SB == 1 ? Layout<4, 1>::kPitch : Layout<4, 2>::kPitch;
}

}  // namespace

GemvFmtPlan gemv_fmt_plan(int M, int64_t N, int64_t K, int r, int log2_block, int num_sms) {
    int G, SB;
    shape_of(log2_block, K, &G, &SB);
    const int tiles = (M * G + 7) / 8;
    const int rows = tiles > 4 ? 16 : 32;                    // row_groups x 16
    const int64_t chunks = (K + 127) / 128;
    // widest slice whose activations fit beside the rest
    int64_t fit = 2;
    while (fit + 2 <= 4096 && plan_smem(M, static_cast<int>(fit + 2), pitch_of(G, SB), rows).total <= kSmemLimit) fit += 2;
    int64_t splits = (chunks + fit - 1) / fit;
    // few rows: more slices, as long as every warp keeps a whole step
    const int64_t by_rows = std::max<int64_t>(1, (N + 15) / 16);
    while (by_rows * splits * 2 <= num_sms && chunks / (splits * 2) >= 2 * kWarps) splits *= 2;
    GemvFmtPlan p;
    int64_t per = (chunks + splits - 1) / splits;
    per = (per + 1) / 2 * 2;
    p.chunks = static_cast<int>(per);
    p.splits = static_cast<int>((chunks + per - 1) / per);
    const int64_t ctas = std::max<int64_t>(1, num_sms / p.splits);
    p.ctas = static_cast<int>(std::min<int64_t>(ctas, by_rows));
    p.warps_k = 1;
    while (p.warps_k < kWarps && p.warps_k * 2 <= (p.chunks + 1) / 2) p.warps_k *= 2;
    p.rows = rows;
    // T's shares: as many CTAs as keep the finalize's reads of their partials short
    const int64_t by_read = 8192 / std::max<int64_t>(1, int64_t(M) * std::max(r, 1) * p.splits);
    p.t_ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(p.ctas, by_read)));
    return p;
}

cudaError_t launch_gemv_fmt(GemvFmtArgs a, const GemvFmtPlan& p, cudaStream_t s) {
    int G, SB;
    shape_of(a.log2_block, a.K, &G, &SB);
    const int tiles = (a.M * G + 7) / 8;
    const int gran = G == 1 ? 128 : G == 2 ? 64 : 32 / SB;
    a.chunks = p.chunks;
    a.warps_k = p.warps_k;
    a.t_ctas = p.t_ctas;
    // 4 consecutive scales at a time, where each is a block of its own and
    // every row and slice begins on a multiple of 4 of them
    a.vec_scales = (1 << a.log2_block) == gran && (a.K / gran) % 4 == 0 && G > 1;
    const int smem = plan_smem(a.M, p.chunks, pitch_of(G, SB), p.rows).total;
    const dim3 grid(static_cast<unsigned>(p.ctas), static_cast<unsigned>(p.splits));
    if (G == 1) return run_tiles<1, 1>(tiles, a, grid, smem, s);
    if (G == 2) return run_tiles<2, 1>(tiles, a, grid, smem, s);
    return SB == 1 ? run_tiles<4, 1>(tiles, a, grid, smem, s) : run_tiles<4, 2>(tiles, a, grid, smem, s);
}

}  // namespace qnf4
