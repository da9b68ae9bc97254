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
//   codes        times a factor (1, 3, 5, 7 or 15, and a power of two) that
//                makes their f16 rounding smallest: FP4 and INT4 are exact,
//                an NF4 code is off by 2^-11 of itself at most, where the
//                bf16 rounding of Y allows 2^-8.
//   activations  times a power of two per token that puts the token's largest
//                value in [2^14, 2^15): their 8 bits are exact in f16 down to
//                2^-28 of the largest; below, off by half a step of the f16
//                subnormals, 2^-25 or 2^-39 of the largest.  The power is 2^126
//                at most; where that is too little, for tokens below 2^-112,
//                every value is exact, a multiple of 2^-133 2^126.
// Both factors are taken out of the sums at the end.
//
// A CTA per SM, 16 warps, each on 32 rows and a share of the contraction, in
// chunks of 128 columns, two to a step.
//   weights      from HBM to registers, 16 bytes (32 weights) per lane and
//                load, the next two chunks in flight while the current ones
//                are multiplied.  Lane (g, c) holds rows g and g + 8 of a
//                16-row group, columns 32 c ... 32 c + 31 of the chunk.
//                Reading a 117 MB weight this way and nothing else takes 21.0
//                us; through rings in shared memory (cp.async, TMA) 20.7, but
//                then the second pass over the packed words competes with the
//                table's for the shared-memory pipe.
//   shared memory  as little as the work allows, since what it leaves is L1,
//                which the weight loads in flight need: 28672 x 8192 with one
//                token took 47 us with 227 KiB reserved, 41 with 130.
//   products     mma.sync m16n8k16, W rows on the M side, tokens on the N
//                side; the contraction order is permuted alike on both
//                operands.  The four lanes of a row hold weights of up to four
//                blocks, which one MMA must not add up:
//                - few tokens: the MMA's 8 columns are (token, block) pairs,
//                  holding x where the lane's weights are of that block and
//                  zero elsewhere, so that each column sums one block;
//                - more tokens: the lanes of a row exchange words (shuffles)
//                  until each holds a quarter of every block.
//   expansion    a packed byte addresses a pair of f16 codes in a table with
//                a copy per lane (no bank conflicts): one byte permute and
//                one 4-byte shared load per two weights, no arithmetic.
//   scales       as stored (codes or fp32) copied to shared memory once for
//                many rows, along the rows; a warp decodes its rows' scales of
//                a step to fp32, a row a lane, just before it uses them.
//                (Loaded from global memory a row a lane: 32 lines per load.)
//   joining      no barrier but one per span of rows (all of the CTA's where
//                they fit): the warps leave their sums in shared memory, and
//                then a thread per output adds them in warp order, with the
//                LoRA term gamma T B^T (T = X A^T from lora_t_kernel, which
//                runs beside the start of this one).  A barrier for every 32
//                rows cost 10 us.  Contraction slices, taken where a CTA's
//                activations would not fit, or with several tokens would leave
//                little L1, write partial sums that join_slices_kernel adds.
// Bound: no unit, but the 16 warps' latencies.
//   1 token (28672 x 8192): about the sum of reading the packed words alone,
//   21.0 us, and of lookups and products alone on words already in registers,
//   16.5 us (81 cycles per 4096 weights).  The two overlap little: a warp asks
//   for a chunk's successor when it has used the chunk up, and 194 rows a CTA
//   are 6 groups of 32 and one of 2 for the 8 groups of warps.  The busiest
//   unit is the shared-memory and L1 pipe, at 66% of its peak (for 4096 weights
//   64 wavefronts of table loads, and the 2 KiB of packed words from L2 pass
//   through it too); DRAM 38%.
//   16 tokens (8192 x 28672): that pipe 49%, issue slots 47%, DRAM 22%, tensor
//   cores 21%.  The warps wait for fixed-latency results and shared loads,
//   four of them a scheduler; a CTA's 683 rows are units of 256 in spans with
//   a barrier between, and each slice's 12 CTAs convert the same activations.
// Registers: instances with exchanged words spill, one tile 4 bytes a thread
// (blocks of 16) to 24 (32), two tiles 16 (16), 44 (32; 64 with fp32 scales) and
// 92 (64 with 8-bit scales); the others do not.
// Measured (us; % of a 6568 GB/s copy on packed words and scales):
//   28672 x 8192, NF4, blocks of 64, E4M3 scales: 37.3 with 1 token (50%),
//   43.2 with 4, 56.2 with 8, 90.8 with 16; with rank 16, 1 token, 38.4
//   28672 x 8192, NF4, blocks of 16, fp32 scales: 64.3 with 1 token, 134 with 16
//   8192 x 28672, INT4, blocks of 128, fp32 scales: 38.8 with 1 token, 72.3 with 16
//   11008 x 4096, NF4, blocks of 32, U8 scales, rank 64, 4 tokens: 20.5
//   4096 x 4096, FP4, blocks of 16, E4M3 scales, 1 token: 7.2; NF4, blocks of 64: 6.6
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "kernels.cuh"

namespace qnf4 {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kSmemSmall = 163 * 1024;       // leaves 92 KiB of L1: the weight loads in flight need it
constexpr int kLutBytes = 256 * 256;         // 256 byte values, 64 words apart, 32 lanes' copies
constexpr int kRows = 32;                    // rows of a warp
constexpr int kCols = 256;                   // columns of a step

// Shared-memory plan, in shared-space addresses.  The code table comes first,
// at a constant, so that a lane's address in it is a byte of its word dropped
// into bits 8-15 of the lane's number times 4, and needs no addition.  Its
// entries use half of their 256 bytes; the first tokens' activations sit in
// the other halves.  Then the other tokens' activations, a line of zeros,
// staged scales, partial sums, T, the tokens' largest magnitudes and factors.
// Dynamic shared memory begins where the driver's own part (1 KiB) ends; the
// plan uses none of the first kReserved bytes.
constexpr uint32_t kReserved = 2048, kLut = kReserved;
struct Plan {
    int unit_rows, span_rows, x_pitch, hole_tokens;
    int raw_pitch, meta_pitch, scale_pitch, red_pitch;    // words (scale_pitch: fp32 of a row in a step)
    uint32_t x, zero, raw, meta, scales, red, t, misc;
    int64_t total;
};

// What the plan follows from: tokens, 128-wide chunks of a slice, columns that
// share a scale, rank, log2 of the block, fp32 scales, warps along the
// contraction, and units of rows per span.
struct PlanKey {
    int M, chunks, gran, r, log2_block, f32, warps_k, span;
};

// fp32 of a row's scales of a step in a warp's area: pitches at which 8 rows'
// loads of a chunk's entries meet no bank twice.
__host__ __device__ constexpr int scale_pitch(int gran) { return gran == 128 ? 2 : gran == 64 ? 6 : 256 / gran + 4; }

inline Plan plan_smem(const PlanKey& k) {
    Plan p;
    p.unit_rows = kRows * (kWarps / k.warps_k);
    p.span_rows = k.span * p.unit_rows;
    p.total = kLut + kLutBytes;
    auto take = [&](int64_t bytes) {
        const uint32_t at = static_cast<uint32_t>(p.total);
        p.total += (bytes + 127) / 128 * 128;
        return at;
    };
    p.x_pitch = ((k.chunks + 1) / 2 * 2) * 256;
    p.hole_tokens = 256 * 128 / p.x_pitch < k.M ? 256 * 128 / p.x_pitch : k.M;
    // a row's stored scales in the slice, and the words that hold them at any
    // alignment; odd pitches, so that a row a lane meets no bank twice
    const int blocks = ((k.chunks * 128) >> k.log2_block) + 2;
    p.raw_pitch = (k.f32 ? blocks : blocks / 4 + 2) | 1;
    p.meta_pitch = k.f32 ? 0 : (blocks / 256 + 2) | 1;
    p.scale_pitch = scale_pitch(k.gran);
    p.red_pitch = k.warps_k + 1;
    p.scales = take(kWarps * kRows * p.scale_pitch * 4);
    p.t = take(k.M * k.r * 4);
    p.misc = take(2 * 16 * 4);
    p.zero = take(128);
    p.x = take(int64_t(k.M - p.hole_tokens) * p.x_pitch);
    p.red = take(int64_t(k.M) * p.span_rows * p.red_pitch * 4);
    p.raw = take(int64_t(p.span_rows) * p.raw_pitch * 4);
    p.meta = take(int64_t(p.span_rows) * p.meta_pitch * 4);
    return p;
}

// 16 bytes where `in`, else v stays: rows and columns outside give sums that
// are not stored, or meet zero activations.
__device__ __forceinline__ void ldg_weights(uint4& v, const uint8_t* p, bool in) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w) : "l"(p), "r"(static_cast<int>(in)));
}
// The table entry at an offset.  Not volatile, so that the compiler may order
// lookups freely; what keeps them behind the barrier that completes the table
// is their address, made of packed words that are loaded after it (by volatile
// assembly) or, the first step's, pass through after_barrier.
__device__ __forceinline__ uint32_t lds_table(uint32_t addr) {
    uint32_t v;
    asm("ld.shared.b32 %0, [%1 + %2];" : "=r"(v) : "r"(addr), "n"(kLut));
    return v;
}

// Makes v known only from this point of the program on; no instruction.  (Done
// to the lane's number in the address instead, it cost a register over the
// whole loop: 28672 x 8192, 16 tokens, 90.8 us, so 92.9.)
__device__ __forceinline__ void after_barrier(uint4& v) {
    asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)::"memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zero.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// kGran: columns that share a scale, up to a chunk.  kCol: (token, block)
// columns, else exchanged words.  NT: tiles of 8 tokens (1 with kCol).
template <int kGran, bool kCol, int NT, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
gemv_fmt_kernel(const __grid_constant__ GemvFmtArgs a, const __grid_constant__ Plan p) {
    constexpr int kPer = 128 / kGran;                     // scales of a row and chunk
    constexpr int E = kCols / kGran;                      // of a step
    constexpr int kPitch = scale_pitch(kGran);
    constexpr int G = !kCol || kGran == 128 ? 1 : kGran == 64 ? 2 : 4;     // columns per token
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* const at0 = smem - smem_u32(smem);           // shared-space address to generic
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    launch_dependents();

    const int64_t K = a.K;
    const int M = a.M;
    const int64_t k_beg = int64_t(blockIdx.y) * a.chunks * 128;
    const int kslab = static_cast<int>(min(K - k_beg, int64_t(a.chunks) * 128));
    float* const scales = reinterpret_cast<float*>(at0 + p.scales) + warp * kRows * kPitch;
    uint32_t* const smax = reinterpret_cast<uint32_t*>(at0 + p.misc);
    float* const sundo = reinterpret_cast<float*>(at0 + p.misc + 64);

    // rows of this CTA, and this warp's part of a unit: 32 rows (the wr-th
    // such group of the unit) x steps m0 ... m1 - 1
    // (no division here: the first loads wait for these)
    const int64_t r0 = blockIdx.x * a.rows + min(int64_t(blockIdx.x), a.extra);
    const int64_t r1 = r0 + a.rows + (int64_t(blockIdx.x) < a.extra ? 1 : 0);
    const int warps_k = 1 << a.log2_warps, unit_rows = p.unit_rows;
    const int wk = warp & (warps_k - 1), wr = warp >> a.log2_warps;
    const int units = static_cast<int>(r1 - r0 + unit_rows - 1) >> (9 - a.log2_warps);      // 32 x 16 rows / warps_k
    const int steps = (kslab + kCols - 1) / kCols;
    const int m0 = steps * wk >> a.log2_warps, m1 = steps * (wk + 1) >> a.log2_warps;
    auto rows_in = [&](int u) {
        const int64_t left = r1 - (r0 + int64_t(u) * unit_rows + wr * kRows);
        return static_cast<int>(min(left, int64_t(kRows)));
    };

    // The weight stream runs a step ahead of the products: (lu, lm) is the
    // step it takes next, wp[i] this lane's words of row 8 i + g there.
    uint4 buf[2][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) buf[i >> 2][i & 3] = make_uint4(0u, 0u, 0u, 0u);
    int lu = 0, lm = m0, lrows = 0;
    const uint8_t* wp[4];
    auto seek_weights = [&]() {
        const int64_t n = r0 + int64_t(lu) * unit_rows + wr * kRows + g;
        lrows = rows_in(lu) - g;
        wp[0] = a.packed + ((n * K + k_beg + m0 * kCols) >> 1) + c * 16;
#pragma unroll
        for (int i = 1; i < 4; ++i) wp[i] = wp[i - 1] + 4 * K;
    };
    auto load_chunk = [&](int cc) {
        const bool in = lm * kCols + cc * 128 + c * 32 < kslab;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ldg_weights(buf[cc][i], wp[i] + cc * 64, in && 8 * i < lrows);
        }
    };
    auto next_step = [&]() {
        if (++lm < m1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) wp[i] += kCols / 2;
        } else {
            lm = m0;
            if (++lu < units) seek_weights();
        }
    };
    // the first loads travel while the table and the activations are set up
    if (m0 < m1 && units > 0) {
        seek_weights();
        load_chunk(0);
        load_chunk(1);
        next_step();
    }

    // Stored scales of the span's rows from row n0 on: a warp per row, the
    // words that hold the slice's blocks b0 ... b1, and their groups'
    // constants.
    auto copy_scales = [&](int64_t n0) {
        const int64_t all = (a.N * K + (int64_t(1) << a.log2_block) - 1) >> a.log2_block;
        for (int row = warp; row < p.span_rows && n0 + row < r1; row += kWarps) {
            const int64_t f = (n0 + row) * K + k_beg;
            const int64_t b0 = f >> a.log2_block, b1 = (f + kslab - 1) >> a.log2_block;
            const uint32_t raw = p.raw + row * p.raw_pitch * 4;
            if (kF32) {
                const float* src = static_cast<const float*>(a.scales) + b0;
                for (int w = lane; w <= b1 - b0; w += 32) cp_async4(raw + w * 4, src + w, 4);
            } else {
                const int64_t w0 = b0 & ~int64_t(3);
                const uint8_t* src = static_cast<const uint8_t*>(a.scales) + w0;
                for (int w = lane; w0 + 4 * w <= b1; w += 32)
                    cp_async4(raw + w * 4, src + 4 * w, static_cast<int>(min(all - (w0 + 4 * w), int64_t(4))));
                const uint32_t meta = p.meta + row * p.meta_pitch * 4;
                for (int w = lane; w <= (b1 >> 8) - (b0 >> 8); w += 32) cp_async4(meta + w * 4, a.meta + (b0 >> 8) + w, 4);
            }
        }
    };
    copy_scales(r0);
    cp_async_commit();

    // code table: byte e of lane l at 256 e + 4 l
    for (int i = tid; i < 256 * 8; i += kThreads) {
        const int e = i >> 3;
        const uint32_t v = a.code[e & 15] | (uint32_t(a.code[e >> 4]) << 16);
        *reinterpret_cast<uint4*>(at0 + kLut + e * 256 + (i & 7) * 16) = make_uint4(v, v, v, v);
    }
    // activations: each token's largest finite magnitude, then f16 copies
    // scaled by it, zeros past the slice, in the order of the MMAs: 16-byte
    // word (pair of MMAs m2, lane c) of a chunk holds that lane's four
    // columns of either MMA.  A chunk is two pieces of 128 bytes (m2 / 2), a
    // piece two words of 64 (m2 & 1, exchanged for odd tokens, so that two
    // tokens' loads share no bank).
    if (tid < 16) smax[tid] = 0;
    if (tid < 8) *reinterpret_cast<uint4*>(at0 + p.zero + tid * 16) = make_uint4(0u, 0u, 0u, 0u);
    auto x_base = [&](int m) {                              // token m's first piece, and the pieces' stride
        return m < p.hole_tokens ? make_int2(kLut + m * (p.x_pitch / 128) * 256 + 128, 256)
                                 : make_int2(p.x + (m - p.hole_tokens) * p.x_pitch, 128);
    };
    __syncthreads();
    const int words = steps * (kCols / 8);                  // 16-byte words per token
    const uint4* const xs = reinterpret_cast<const uint4*>(a.X + k_beg);
    constexpr int kAhead = kCol ? 1 : 4;                               // words of a thread in flight
    const int all_words = M * words;
    uint4 xv[kAhead];
    auto for_words = [&](bool fetch, auto use) {            // use(token, word, its value); the token is uniform in a
        for (int base = tid; base < all_words; base += kAhead * kThreads) {        // warp: 32 | words
            int m[kAhead], w[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int at = base + i * kThreads;
                m[i] = M == 1 ? 0 : at / words;
                w[i] = at - m[i] * words;
                if (fetch) {
                    xv[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (at < all_words && w[i] * 8 < kslab) xv[i] = __ldg(xs + m[i] * (K / 8) + w[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (base + i * kThreads < all_words) use(m[i], w[i], xv[i]);
        }
    };
    for_words(true, [&](int m, int, const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t mx = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t lo = w[q] & 0x7fffu, hi = (w[q] >> 16) & 0x7fffu;
            if (lo < 0x7f80u) mx = max(mx, lo);
            if (hi < 0x7f80u) mx = max(mx, hi);
        }
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (lane == 0) atomicMax(smax + m, mx);
    });
    __syncthreads();
    for_words(all_words > kAhead * kThreads, [&](int m, int w, const uint4& v) {
        const int sh = min(126, 14 + 127 - static_cast<int>(smax[m] >> 7));
        const float f = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
        const uint32_t in[4] = {v.x, v.y, v.z, v.w};
        uint32_t out[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const __half2 h = __floats2half2_rn(__uint_as_float(in[q] << 16) * f,
                                                __uint_as_float(in[q] & 0xffff0000u) * f);
            out[q] = *reinterpret_cast<const uint32_t*>(&h);
        }
        const uint4 o = make_uint4(out[0], out[1], out[2], out[3]);
        // columns 8 u ... 8 u + 7 of the chunk: where in it
        const int u = w & 15;
        constexpr bool kWhole = kCol || kGran == 128;       // lane c: columns 32 c ... 32 c + 31
        const int m2 = kWhole ? u & 3 : kGran == 64 ? (u >> 3) * 2 + (u & 1) : u >> 2;
        const int2 xb = x_base(m);
        uint8_t* at = at0 + xb.x + (w >> 4) * 2 * xb.y + (m2 >> 1) * xb.y + ((m2 ^ m) & 1) * 64;
        // exchanged words: quarter q of a run of 64 or 16 sits in lane
        // 0, 2, 1, 3 for q = 0 ... 3
        if (kWhole || kGran >= 32) {
            const int q = (u >> 1) & 3;
            const int cl = kWhole ? u >> 2 : kGran == 64 ? ((q & 1) << 1) | (q >> 1) : u & 3;
            *reinterpret_cast<uint4*>(at + cl * 16) = o;
        } else {
            // blocks of 16: quarters 2 (u & 1) and the next, for the pair's
            // first or second MMA
            at += (u & 1) * 16 + ((u >> 1) & 1) * 8;
            *reinterpret_cast<uint2*>(at) = make_uint2(o.x, o.y);
            *reinterpret_cast<uint2*>(at + 32) = make_uint2(o.z, o.w);
        }
        if (w == 0) sundo[m] = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
    });
    cp_async_wait<0>();                                     // the scales
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) after_barrier(buf[i >> 2][i & 3]);

    // This lane's column of each tile: its token's activations, with (token,
    // block) columns only where the lane's weights are of the column's block;
    // elsewhere zeros (left in place with one tile, read from a line of them
    // with two).
    uint32_t xoff[NT], xpiece[NT];
    bool xon = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int tok = (8 * t + g) / G;
        xon = tok < M && (G == 1 || g % G == (G == 2 ? c >> 1 : c));
        const int2 xb = x_base(xon ? tok : 0);
        xoff[t] = (xon ? xb.x : p.zero) + (tok & 1) * 64 + c * 16;
        xpiece[t] = xon ? xb.y : 0;
    }
    uint4 x1[4];
#pragma unroll
    for (auto& v : x1) v = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t lane4 = lane * 4;
    auto code_pair = [&](uint32_t w, uint32_t sel) { return lds_table(prmt(w, lane4, sel)); };
    constexpr int kTok = G == 1 ? 4 : 2;                  // totals per tile: two tokens' or one's, of two rows
    float tot[2][NT][kTok];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < kTok; ++e) tot[q][t][e] = 0.f;

    // One row's words of a chunk, exchanged among the row's four lanes.
    auto exchange = [&](const uint4& v, uint32_t (&w)[4]) {
        if (kCol || kGran == 128) {
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            return;
        }
        // halves with lane c ^ 2: first runs' words (w0, w1), then the others
        const bool up = c & 2;
        const uint32_t r0w = __shfl_xor_sync(0xffffffffu, up ? v.x : v.z, 2), r1w = __shfl_xor_sync(0xffffffffu, up ? v.y : v.w, 2);
        w[0] = up ? r0w : v.x;
        w[1] = up ? r1w : v.y;
        w[2] = up ? v.z : r0w;
        w[3] = up ? v.w : r1w;
        if (kGran == 64) return;
        // words with lane c ^ 1: word c of each of the four 16-byte units
        const bool odd = c & 1;
        const uint32_t s0 = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1), s1 = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
        const uint32_t a0 = odd ? s0 : w[0], a1 = odd ? w[1] : s0, a2 = odd ? s1 : w[2], a3 = odd ? w[3] : s1;
        w[0] = a0; w[1] = a1; w[2] = a2; w[3] = a3;
        if (kGran == 32) return;
        // half words with lane c ^ 2: two bytes of each block of 16
        const uint32_t h0 = __shfl_xor_sync(0xffffffffu, prmt(w[0], w[1], up ? 0x5410u : 0x7632u), 2);
        const uint32_t h1 = __shfl_xor_sync(0xffffffffu, prmt(w[2], w[3], up ? 0x5410u : 0x7632u), 2);
        // lower lanes: own low half, then the other's low half; upper lanes:
        // the other's high half, then the own high half
        w[0] = up ? prmt(h0, w[0], 0x7610u) : prmt(w[0], h0, 0x5410u);
        w[1] = up ? prmt(h0, w[1], 0x7632u) : prmt(w[1], h0, 0x7610u);
        w[2] = up ? prmt(h1, w[2], 0x7610u) : prmt(w[2], h1, 0x5410u);
        w[3] = up ? prmt(h1, w[3], 0x7632u) : prmt(w[3], h1, 0x7610u);
    };

    // Chunk cc of the current step, in buf[cc]: NQ 16-row groups; ch, the
    // chunk within the slice.
    auto chunk = [&](auto nq, int cc, int ch) {
        constexpr int NQ = decltype(nq)::value;
        uint32_t xa[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xa[t] = xoff[t] + 2 * ch * xpiece[t];
        if (NT == 1) {
#pragma unroll
            for (int m2 = 0; m2 < 4; ++m2)
                if (xon) x1[m2] = *reinterpret_cast<const uint4*>(at0 + ((xa[0] + (m2 >> 1) * xpiece[0]) ^ ((m2 & 1) * 64u)));
        }
        float d[NQ][NT][4];
        uint32_t w[NQ][2][4];
#pragma unroll
        for (int i = 0; i < 2 * NQ; ++i) exchange(buf[cc][i], w[i >> 1][i & 1]);
        // MMAs 4 b ... that share the sets of blocks: kGran / 16 of them, or
        // with (token, block) columns the lane's 32 weights, 16 at a time for
        // blocks of 16
        constexpr int kRun = kCol ? (kGran == 16 ? 4 : 8) : kGran / 16;
        uint4 x[NT];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t lo = 0x7604u | (j & 1) << 5, hi = lo | 1u << 4;     // bytes 2 (j & 1) and the next
            const int m2 = j >> 1;
            if (NT == 1) {
                x[0] = x1[m2];
            } else if ((j & 1) == 0) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    x[t] = *reinterpret_cast<const uint4*>(at0 + ((xa[t] + (m2 >> 1) * xpiece[t]) ^ ((m2 & 1) * 64u)));
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const uint32_t a0 = code_pair(w[q][0][m2], lo), a1 = code_pair(w[q][1][m2], lo);
                const uint32_t a2 = code_pair(w[q][0][m2], hi), a3 = code_pair(w[q][1][m2], hi);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t b0 = j & 1 ? x[t].z : x[t].x, b1 = j & 1 ? x[t].w : x[t].y;
                    if (j % kRun == 0) mma_f16_first(d[q][t], a0, a1, a2, a3, b0, b1);
                    else mma_f16(d[q][t], a0, a1, a2, a3, b0, b1);
                }
            }
            if (j % kRun == kRun - 1) {
                // the blocks' sums times their scales
                const int run = j / kRun;
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    const float* sr = scales + (q * 16 + g) * kPitch + cc * kPer;
                    const float* sr8 = sr + 8 * kPitch;
                    if constexpr (G == 1) {               // two tokens, one block
                        const float s0 = sr[run], s1 = sr8[run];
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            tot[q][t][0] = fmaf(s0, d[q][t][0], tot[q][t][0]);
                            tot[q][t][1] = fmaf(s0, d[q][t][1], tot[q][t][1]);
                            tot[q][t][2] = fmaf(s1, d[q][t][2], tot[q][t][2]);
                            tot[q][t][3] = fmaf(s1, d[q][t][3], tot[q][t][3]);
                        }
                    } else {                              // one token, two blocks: b and b + step
                        const int b = G == 2 ? 0 : kGran == 32 ? 2 * (c & 1) : 4 * (c & 1) + run;
                        constexpr int step = kGran == 16 ? 2 : 1;
                        tot[q][0][0] = fmaf(sr[b], d[q][0][0], fmaf(sr[b + step], d[q][0][1], tot[q][0][0]));
                        tot[q][0][1] = fmaf(sr8[b], d[q][0][2], fmaf(sr8[b + step], d[q][0][3], tot[q][0][1]));
                    }
                }
            }
        }
    };

    // Row `lane` of the warp's rows in the current unit: its stored scales,
    // and where in its first block the slice begins.
    uint32_t lraw = 0, lmeta = 0;
    int lfirst = 0, lb0 = 0;
    auto seek_scales = [&](int64_t n, int span_row) {
        const int64_t f = n * K + k_beg, b0 = f >> a.log2_block;
        lfirst = static_cast<int>(f & ((int64_t(1) << a.log2_block) - 1));
        lb0 = static_cast<int>(b0 & 255);
        lraw = p.raw + span_row * p.raw_pitch * 4 + (kF32 ? 0 : static_cast<int>(b0 & 3));
        lmeta = p.meta + span_row * p.meta_pitch * 4;
    };
    // Its scales of a step to fp32 in this warp's area.
    auto decode_scales = [&](int mi) {
        float v[E];
        const int i0 = (lfirst + mi * kCols) >> a.log2_block;        // the first one's block, from b0 on
        if (kF32) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = a.vec_scales ? i0 + e : (lfirst + min(mi * kCols + e * kGran, kslab - kGran)) >> a.log2_block;
                v[e] = *reinterpret_cast<const float*>(at0 + lraw + i * 4);
            }
        } else if (a.vec_scales) {                        // E blocks in a row, in one word each four, in one group
            const float m = *reinterpret_cast<const float*>(at0 + lmeta + ((lb0 + i0) >> 8) * 4);
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const uint32_t w = E >= 4 ? *reinterpret_cast<const uint32_t*>(at0 + lraw + i0 + e)
                                          : *reinterpret_cast<const uint16_t*>(at0 + lraw + i0);
                if (a.scale_fmt == QLORA_SCALES_E4M3) {
#pragma unroll
                    for (int q = 0; q < (E < 4 ? E : 4); q += 2) {
                        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                            static_cast<__nv_fp8x2_storage_t>(w >> (8 * q)), __NV_E4M3);
                        const float2 f = __half22float2(__half2(h));
                        v[e + q] = __fmul_rn(f.x, m);
                        v[e + q + 1] = __fmul_rn(f.y, m);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < (E < 4 ? E : 4); ++q) {
                        const uint32_t code = (w >> (8 * q)) & 0xffu;
                        v[e + q] = __fmul_rn(a.scale_fmt == QLORA_SCALES_U8 ? static_cast<float>(code)
                                                                            : e5m2_to_float(static_cast<uint8_t>(code)), m);
                    }
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                // columns past the slice repeat its last scale
                const int i = (lfirst + min(mi * kCols + e * kGran, kslab - kGran)) >> a.log2_block;
                const uint32_t code = at0[lraw + i];
                const float m = *reinterpret_cast<const float*>(at0 + lmeta + ((lb0 + i) >> 8) * 4);
                v[e] = __fmul_rn(a.scale_fmt == QLORA_SCALES_U8 ? static_cast<float>(code)
                                 : a.scale_fmt == QLORA_SCALES_E4M3 ? e4m3_to_float(static_cast<uint8_t>(code))
                                                                    : e5m2_to_float(static_cast<uint8_t>(code)), m);
            }
        }
        float* at = scales + lane * kPitch;
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(at + e) = make_float2(v[e], v[e + 1]);
    };

    // The steps of this warp's rows in a unit.  (A chunk past the slice has
    // zero activations.)
    auto run_unit = [&](auto nq, int rows) {
        for (int mi = m0; mi < m1; ++mi) {
            const bool more = lu < units;
            if (lane < rows) decode_scales(mi);
            __syncwarp();
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                chunk(nq, cc, 2 * mi + cc);
                if (more) load_chunk(cc);
            }
            if (more) next_step();
            __syncwarp();                                 // the step's scales have been used
        }
    };
    auto skip_unit = [&]() {
        for (int mi = m0; mi < m1 && lu < units; ++mi) {
            load_chunk(0);
            load_chunk(1);
            next_step();
        }
    };

    float* const red = reinterpret_cast<float*>(at0 + p.red);
    float* const sT = reinterpret_cast<float*>(at0 + p.t);
    for (int u0 = 0; u0 < units; u0 += a.span) {
        const int64_t n0 = r0 + int64_t(u0) * unit_rows;  // the span's first row
        if (u0 > 0) {
            copy_scales(n0);
            cp_async_commit();
            cp_async_wait<0>();
            __syncthreads();
        }
        const int u1 = min(units, u0 + a.span);
        for (int u = u0; u < u1; ++u) {
            const int rows = rows_in(u);
            const int span_row = (u - u0) * unit_rows + wr * kRows;
            seek_scales(n0 + span_row + lane, span_row + lane);
            // straight-line steps of either height, so that a chunk's lookups
            // overlap the products of the one before
            if (rows > 16) run_unit(std::integral_constant<int, 2>{}, rows);
            else if (rows > 0) run_unit(std::integral_constant<int, 1>{}, rows);
            else skip_unit();
            // partial sums [token][row][warp]
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float* const row = red + (span_row + q * 16 + g) * p.red_pitch + wk;
                    const int tok_stride = p.span_rows * p.red_pitch;
                    if constexpr (G == 1) {
                        const int tok = 8 * t + 2 * c;
                        if (tok < M) {
                            row[tok * tok_stride] = tot[q][t][0];
                            row[tok * tok_stride + 8 * p.red_pitch] = tot[q][t][2];
                        }
                        if (tok + 1 < M) {
                            row[(tok + 1) * tok_stride] = tot[q][t][1];
                            row[(tok + 1) * tok_stride + 8 * p.red_pitch] = tot[q][t][3];
                        }
                    } else {
                        float v0 = tot[q][t][0], v1 = tot[q][t][1];
                        if (G == 4) {                     // the token's other two blocks
                            v0 += __shfl_xor_sync(0xffffffffu, v0, 1);
                            v1 += __shfl_xor_sync(0xffffffffu, v1, 1);
                        }
                        const int tok = G == 2 ? c : c >> 1;
                        if (tok < M && (G == 2 || (c & 1) == 0)) {
                            row[tok * tok_stride] = v0;
                            row[tok * tok_stride + 8 * p.red_pitch] = v1;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < kTok; ++e) tot[q][t][e] = 0.f;
                }
        }
        if (u0 == 0 && a.t_rank > 0) {
            grid_dependency_wait();                       // T is complete
            for (int i = tid; i < M * a.t_rank; i += kThreads) sT[i] = a.T[i];
        }
        __syncthreads();                                  // all partial sums are there
        const int rows = static_cast<int>(min(int64_t(p.span_rows), r1 - n0));
        for (int o = tid; o < M * rows; o += kThreads) {
            const int m = M == 1 ? 0 : o / rows, row = o - m * rows;
            const int64_t n = n0 + row;
            const float* src = red + (m * p.span_rows + row) * p.red_pitch;
            float s = 0.f;
            for (int w = 0; w < warps_k; ++w) s += src[w];
            // in 64 bits: the two factors together, 2^-126 ... 2^113 and 2^-149 ... 2^128,
            // leave fp32's range where the product need not
            s = static_cast<float>(s * (sundo[m] * a.code_undo));
            if (a.part != nullptr) {
                a.part[(int64_t(blockIdx.y) * M + m) * a.N + n] = s;
                continue;
            }
            float l = 0.f;
#pragma unroll 2
            for (int j = 0; j < a.t_rank; j += 8) {
                const uint4 bv = __ldg(reinterpret_cast<const uint4*>(a.B + n * a.t_rank + j));
                const uint32_t bw[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    l = fmaf(sT[m * a.t_rank + j + 2 * q], __uint_as_float(bw[q] << 16), l);
                    l = fmaf(sT[m * a.t_rank + j + 2 * q + 1], __uint_as_float(bw[q] & 0xffff0000u), l);
                }
            }
            const __nv_bfloat16 y = __float2bfloat16_rn(fmaf(a.gamma, l, s));
            a.Y[m * a.N + n] = *reinterpret_cast<const uint16_t*>(&y);
        }
        if (u1 < units) __syncthreads();                  // sums and scales have been read
    }
    // the joining kernel, this one's dependent, reads T too
    if (a.part != nullptr) grid_dependency_wait();
}

// T[m][j] = x[m] . A[j] in fp32: a CTA per rank and kM tokens (all 16 in one
// CTA took 12 us at 4096 columns), its warps on equal runs of the contraction,
// added in warp order.
constexpr int kTThreads = 512;
template <int kM>
__global__ void __launch_bounds__(kTThreads)
lora_t_kernel(const uint16_t* __restrict__ X, const uint16_t* __restrict__ A, float* __restrict__ T, int M, int64_t K, int r) {
    __shared__ float part[kTThreads / 32][kM];
    launch_dependents();
    const int j = blockIdx.x, mb = blockIdx.y * kM, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n8 = static_cast<int>(K / 8);
    const int s0 = n8 * warp / (kTThreads / 32), s1 = n8 * (warp + 1) / (kTThreads / 32);      // K <= 2^24
    const uint4* const a8 = reinterpret_cast<const uint4*>(A + j * K);
    const uint4* x8[kM];
    float t[kM];
#pragma unroll
    for (int m = 0; m < kM; ++m) {
        x8[m] = reinterpret_cast<const uint4*>(X + min(mb + m, M - 1) * K);
        t[m] = 0.f;
    }
#pragma unroll(kM == 1 ? 4 : 2)
    for (int s = s0 + lane; s < s1; s += 32) {
        const uint4 av = __ldg(a8 + s);
        const uint32_t aw[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            const uint4 xv = __ldg(x8[m] + s);
            const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                t[m] = fmaf(__uint_as_float(aw[e] << 16), __uint_as_float(xw[e] << 16), t[m]);
                t[m] = fmaf(__uint_as_float(aw[e] & 0xffff0000u), __uint_as_float(xw[e] & 0xffff0000u), t[m]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < kM; ++m) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) t[m] += __shfl_xor_sync(0xffffffffu, t[m], o);
        if (lane == 0) part[warp][m] = t[m];
    }
    __syncthreads();
    if (threadIdx.x < kM && mb + threadIdx.x < M) {
        float s = 0.f;
        for (int w = 0; w < kTThreads / 32; ++w) s += part[w][threadIdx.x];
        T[(mb + threadIdx.x) * r + j] = s;
    }
}

// Y[m][n] = bf16(sum of the slices' partial products, in slice order, + gamma
// T[m] . B[n]): a thread per row n and two tokens.
constexpr int kJoinTokens = 2;               // 8192 x 28672, 16 tokens: 71.7 us; with 4 74.7
__global__ void __launch_bounds__(256)
join_slices_kernel(const __grid_constant__ GemvFmtArgs a, int splits) {
    grid_dependency_wait();                               // everything comes from the kernels before
    const int64_t n = blockIdx.x * int64_t(blockDim.x) + threadIdx.x;
    if (n >= a.N) return;
    const int mb = blockIdx.y * kJoinTokens;
    float s[kJoinTokens], l[kJoinTokens];
#pragma unroll
    for (int i = 0; i < kJoinTokens; ++i) {
        s[i] = l[i] = 0.f;
        if (mb + i < a.M) {
            const float* part = a.part + int64_t(mb + i) * a.N + n;
#pragma unroll 4
            for (int k = 0; k < splits; ++k) s[i] += part[int64_t(k) * a.M * a.N];
        }
    }
#pragma unroll 2
    for (int j = 0; j < a.t_rank; j += 8) {
        const uint4 bv = __ldg(reinterpret_cast<const uint4*>(a.B + n * a.t_rank + j));
        const uint32_t bw[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
        for (int i = 0; i < kJoinTokens; ++i) {
            if (mb + i < a.M) {
                const float4* t = reinterpret_cast<const float4*>(a.T + (mb + i) * a.t_rank + j);
                const float4 t0 = t[0], t1 = t[1];
                const float tv[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    l[i] = fmaf(tv[2 * q], __uint_as_float(bw[q] << 16), l[i]);
                    l[i] = fmaf(tv[2 * q + 1], __uint_as_float(bw[q] & 0xffff0000u), l[i]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kJoinTokens; ++i) {
        if (mb + i < a.M) {
            const __nv_bfloat16 y = __float2bfloat16_rn(fmaf(a.gamma, l[i], s[i]));
            a.Y[(mb + i) * a.N + n] = *reinterpret_cast<const uint16_t*>(&y);
        }
    }
}

template <int kGran, bool kCol, int NT, bool kF32>
cudaError_t run(const GemvFmtArgs& a, const Plan& p, dim3 grid, cudaStream_t s) {
    // the plan's addresses hold where dynamic shared memory begins by kReserved
    int dev = 0, reserved = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
    if (e != cudaSuccess) return e;
    if (reserved > static_cast<int>(kReserved)) return cudaErrorInvalidConfiguration;
    // The limit belongs to the kernel, not to the call: set to a plan's size,
    // it would be too low for a larger plan that another host thread is about
    // to launch.
    auto* kernel = gemv_fmt_kernel<kGran, kCol, NT, kF32>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.total);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.t_rank > 0 ? 1 : 0;      // after lora_t_kernel
    return cudaLaunchKernelEx(&cfg, kernel, a, p);
}

template <int kGran, bool kCol, int NT>
cudaError_t run_scales(const GemvFmtArgs& a, const Plan& p, dim3 grid, cudaStream_t s) {
    return a.scale_fmt == QLORA_SCALES_FP32 ? run<kGran, kCol, NT, true>(a, p, grid, s)
                                            : run<kGran, kCol, NT, false>(a, p, grid, s);
}

// (token, block) columns where one tile of 8 holds them all, exchanged words
// beyond (us, columns and exchanged: 28672 x 8192, blocks of 64, 1 token 37.2
// and 41.6, 4 tokens 43.7 and 46.4, 8 tokens in two tiles and one slice 80.6 and 67.7; blocks
// of 16 with fp32 scales, 2 tokens 67.4 and 76.5; 11008 x 4096, blocks of 32, 4
// tokens in two tiles 18.4 and 17.1)
template <int kGran>
cudaError_t run_gran(const GemvFmtArgs& a, const Plan& p, dim3 grid, cudaStream_t s) {
    if constexpr (kGran < 128) {
        if (a.M <= (kGran == 64 ? 4 : 2)) return run_scales<kGran, true, 1>(a, p, grid, s);
    }
    return a.M <= 8 ? run_scales<kGran, false, 1>(a, p, grid, s) : run_scales<kGran, false, 2>(a, p, grid, s);
}

// Columns that share a scale: the block, up to a chunk.  Rows of an odd
// number of 64-wide runs shift a block of 128 or more against the next row's
// chunks by half a chunk, so there each run takes its own scale.
int gran_of(int log2_block, int64_t K) {
    return log2_block <= 6 ? 1 << log2_block : K % 128 != 0 ? 64 : 128;
}

}  // namespace

GemvFmtPlan gemv_fmt_plan(int M, int64_t N, int64_t K, int r, int log2_block, bool f32, int num_sms) {
    const int gran = gran_of(log2_block, K);
    const int64_t chunks = (K + 127) / 128;
    // Slices are whole multiples of 4 chunks: as few as leave their
    // activations the room.
    auto per_of = [&](int64_t splits) { return ((chunks + splits - 1) / splits + 3) / 4 * 4; };
    auto bytes = [&](int64_t splits, int warps_k, int64_t span) {
        return plan_smem({M, static_cast<int>(std::min<int64_t>(per_of(splits), 1 << 20)), gran, r, log2_block, f32, warps_k,
                          static_cast<int>(span)}).total;
    };
    int64_t splits = 1;
    // (several tokens: narrower slices, for the sake of L1; us with slices as
    // wide as shared memory, and so: 28672 x 8192, blocks of 64, 8 tokens 67.7
    // and 56.1, blocks of 16, 4 tokens 91.0 and 80.4; 8192 x 28672, 4 tokens 54.7
    // and 48.5, 16 tokens 79.0 and 71.6; one token has no activations to cut)
    while (per_of(splits) > 4 && bytes(splits, kWarps, 1) > (M > 1 ? kSmemSmall : kSmemLimit)) ++splits;
    // few rows: more slices, as long as every warp keeps a step
    const int64_t by_rows = std::max<int64_t>(1, (N + 15) / 16);
    while (by_rows * splits * 2 <= num_sms && per_of(splits * 2) >= 2 * kWarps) splits *= 2;
    GemvFmtPlan p;
    p.chunks = static_cast<int>(per_of(splits));
    p.splits = static_cast<int>((chunks + p.chunks - 1) / p.chunks);
    p.ctas = static_cast<int>(std::min<int64_t>(std::max<int64_t>(1, num_sms / p.splits), by_rows));
    // warps along the contraction: the least of the busiest warp's steps of
    // 16 rows, and of its units of rows, which cost about two of them (with 16
    // everywhere, 8192 x 28672 with 16 tokens took 149 us, so 108)
    const int64_t rows = (N + p.ctas - 1) / p.ctas, steps = (p.chunks * 128 + kCols - 1) / kCols;
    int64_t best = INT64_MAX;
    p.warps_k = kWarps;
    for (int w = kWarps; w >= 1; w /= 2) {
        if (bytes(splits, w, 1) > kSmemLimit) continue;
        const int64_t unit_rows = kRows * (kWarps / w), full = rows / unit_rows, rest = rows % unit_rows;
        const int64_t cost = (2 * full + (rest > 16 ? 2 : rest > 0)) * ((steps + w - 1) / w) + 2 * (full + (rest > 0));
        if (cost < best) {
            best = cost;
            p.warps_k = w;
        }
    }
    // rows of a CTA in as few equal spans as fit
    const int64_t unit_rows = kRows * (kWarps / p.warps_k), units = (rows + unit_rows - 1) / unit_rows;
    const int64_t limit = std::max<int64_t>(bytes(splits, p.warps_k, 1), kSmemSmall);
    int64_t span = 1;
    while (span < 64 && span < units && bytes(splits, p.warps_k, span + 1) <= limit) ++span;
    const int64_t spans = (units + span - 1) / span;
    p.span = static_cast<int>((units + spans - 1) / spans);
    return p;
}

cudaError_t launch_gemv_fmt(GemvFmtArgs a, const GemvFmtPlan& p, cudaStream_t s) {
    const int gran = gran_of(a.log2_block, a.K);
    if (a.t_rank > 0) {
        auto* kernel = a.M == 1 ? lora_t_kernel<1> : lora_t_kernel<4>;
        kernel<<<dim3(static_cast<unsigned>(a.t_rank), static_cast<unsigned>((a.M + 3) / 4)), kTThreads, 0, s>>>(a.X, a.A, a.T, a.M, a.K, a.t_rank);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    a.chunks = p.chunks;
    a.span = p.span;
    a.log2_warps = 0;
    while ((1 << a.log2_warps) < p.warps_k) ++a.log2_warps;
    a.rows = a.N / p.ctas;
    a.extra = a.N % p.ctas;
    const Plan sp = plan_smem({a.M, p.chunks, gran, a.t_rank, a.log2_block, a.scale_fmt == QLORA_SCALES_FP32, p.warps_k, p.span});
    // a step's scales as whole words of one group, where each is a block of
    // its own and every row begins on a multiple of 4 steps' worth of them
    a.vec_scales = (1 << a.log2_block) == gran && a.K % std::max(kCols, 4 * gran) == 0;
    const dim3 grid(static_cast<unsigned>(p.ctas), static_cast<unsigned>(p.splits));
    const cudaError_t e = gran == 16 ? run_gran<16>(a, sp, grid, s) : gran == 32 ? run_gran<32>(a, sp, grid, s)
                          : gran == 64 ? run_gran<64>(a, sp, grid, s) : run_gran<128>(a, sp, grid, s);
    if (e != cudaSuccess || p.splits == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.N + 255) / 256), static_cast<unsigned>((a.M + kJoinTokens - 1) / kJoinTokens));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_slices_kernel, a, p.splits);
}

}  // namespace qnf4
