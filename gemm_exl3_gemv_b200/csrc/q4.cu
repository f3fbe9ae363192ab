// q4.cu -- products with plain 4-bit weights in groups (exl3_q4_gemm), and
// their packing.
//
//     y[i][n] = sum_k x[i][k] (q[k][n] - z[k/g][n]) s[k/g][n]
//
// This file's kernel takes up to 8 rows, and up to 24 in groups of 32; q4_tc.cu
// takes the others (see takes_tc()).  The product reads half a byte per weight
// and does 2 m flops with it, so at few rows the stream of packed words is the
// bound, if a weight costs less than about three instruction slots (148 SMs x
// 128 lanes at 1.9 GHz against 13e12 weights a second).  Measured, the words'
// and scales' bytes over the time: one row of 5120 x 17408 in groups of 128,
// 13.1 us (3.6 TB/s), of 4096 x 4096 4.3 us, where a launch and the first bytes,
// about 3 us, are the larger part.
//   * The packed tiles (16 channels x 64 inputs, layout in include/exl3.h) are
//     the A operand of mma.m16n8k16 in register order: a lane's 128-bit load
//     is its share of four k-steps, and two fields of a word become an fp16
//     pair by one AND-OR and one packed add: (q - z), an integer below 2048,
//     exact in fp16.  (Taking z sum(x) off the group's sum instead, with the
//     fields as they are, cancels where q is near z: a channel of q = z came
//     out as rounding errors of sum(q x) and not as zero.  It is no faster: one
//     row of 5120 x 17408 12.8 us and 12.9 so, of 17408 x 5120 17.1 and 16.8.)
//   * Words, scales, zero points and x come by asynchronous copies through
//     rings in shared memory: a warp's own for the weights, one shared by the
//     warps that work on the same inputs for x, whose B fragments are 128-bit
//     reads.  (Bulk copies of such small pieces were slower: an SM started one
//     in about 22 ns, and a step needs two to forty of them.)
//   * The fp32 sums of a group are scaled in fp32 and added up; nothing is
//     rounded below 32 bits before the result.
// A warp takes steps of 128 inputs of 16*CT channels; some of a CTA's 8 warps lie
// along the channels, the others along the inputs, and the CTAs of a cut
// (grid.y) split the inputs.  Sums are joined in warp order in shared memory,
// and in CTA order by the last CTA to arrive.
#include <cuda_fp16.h>

#include <type_traits>

#include "exl3_cache.h"
#include "exl3_tc.cuh"

namespace exl3 {

namespace {

constexpr int kQ4MaxDepth = 5;

struct Q4Args {
    const uint16_t* x;
    const uint32_t* packed;
    const uint16_t* scale;
    const uint8_t* zero;
    void* y;
    int m, k_in, n_out, y_fp32;
    int warps_c;              // warps of a CTA along the channels (a power of two; the others along the inputs)
    int splits;               // CTAs that share a channel block's inputs
    int depth;                // stages of the rings
    unsigned char* ws;
    long long part_vecs;      // places of 16 bytes for parts of sums in the workspace (for the debug build's checks)
};

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same into a sum that starts at zero.
__device__ __forceinline__ void mma_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The pair's fields in the mantissa of 1024, in one instruction.
__device__ __forceinline__ __half2 masked_1024(uint32_t w, uint32_t mask)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(mask), "r"(0x64006400u));
    return bits_h2(r);
}

// The A fragment of one k-step: rows g (a0, a2) and g + 8 (a1, a3) of the tile,
// q - z from 1024 + q and 1024 + 16 q: zlo = -(1024 + z), zhi = -(64 + z).
__device__ __forceinline__ void q4_fragment(uint32_t w, __half2 zlo, __half2 zhi, uint32_t (&a)[4])
{
    const uint32_t v = w >> 8;
    const __half2 sixteenth = __float2half2_rn(0.0625f);
    a[0] = h2_bits(__hadd2(masked_1024(w, 0x000F000Fu), zlo));
    a[1] = h2_bits(__hfma2(masked_1024(w, 0x00F000F0u), sixteenth, zhi));
    a[2] = h2_bits(__hadd2(masked_1024(v, 0x000F000Fu), zlo));
    a[3] = h2_bits(__hfma2(masked_1024(v, 0x00F000F0u), sixteenth, zhi));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Reads from shared memory by 32-bit address, so that the compiler adds no
// 64-bit arithmetic to them.
__device__ __forceinline__ uint4 lds16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ float lds_half(uint32_t at)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
    return __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ uint32_t lds_byte(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
// All but the last n groups of this thread's copies have landed.
__device__ __forceinline__ void cp_async_wait(int n)
{
    switch (n) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}

// CT: channel tiles of a warp.  NT: row tiles (of 8).  SPS: steps (of 128
// inputs) that a stage of the rings holds.
template <int CT, int NT, int SPS, int GROUP>
struct Q4Shape {
    static constexpr int kWarps = 8, kThreads = 32 * kWarps;
    static constexpr int kParts = 128 / GROUP;               // groups of a step
    static constexpr int kRows = 8 * NT;
    static constexpr int kScales = SPS * CT * 1024;          // where a stage's scales and zero points lie: per group
    static constexpr int kZeros = kScales + SPS * kParts * CT * 32;
    static constexpr int kStage = kZeros + SPS * kParts * CT * 16;
    static constexpr int kXRow = SPS * 256 + 64;             // bytes from row to row of x: 8 lanes' reads meet no bank twice
    static constexpr int kMinCtas = 2;                       // per SM
};

template <int CT, int NT, int SPS, int GROUP>
__global__ void __launch_bounds__(256, (Q4Shape<CT, NT, SPS, GROUP>::kMinCtas)) q4_gemm_kernel(const __grid_constant__ Q4Args p)
{
    using S = Q4Shape<CT, NT, SPS, GROUP>;
    constexpr int kParts = S::kParts;
    extern __shared__ __align__(128) unsigned char smem[];
    float* red = reinterpret_cast<float*>(smem);             // after the loop: inputs' warps x rows x channels
    __shared__ int last_flag;

    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
    const int wc = warp & (p.warps_c - 1), wk = warp / p.warps_c, warps_k = S::kWarps / p.warps_c;
    const int g = lane >> 2, t = lane & 3;
    const int kt_all = p.k_in / 64, tn_all = p.n_out / 16, steps = (kt_all + 1) / 2;
    const int tn0 = (blockIdx.x * p.warps_c + wc) * CT;
    const int tiles = max(0, min(CT, tn_all - tn0));         // of this warp; the last CTA's may have none
    const int slice = blockIdx.y * warps_k + wk, slices = p.splits * warps_k;
    const int s0 = (int)((long long)steps * slice / slices), s1 = (int)((long long)steps * (slice + 1) / slices);
    const int depth = p.depth;
    unsigned char* ring = smem + warp * depth * S::kStage;
    unsigned char* x_ring = smem + S::kWarps * depth * S::kStage + wk * depth * (p.m * S::kXRow);
    if (!p.zero)                                             // no copy comes there
        for (int i = 0; i < depth; ++i)
            for (int j = 4 * lane; j < S::kStage - S::kZeros; j += 128)
                *reinterpret_cast<uint32_t*>(ring + i * S::kStage + S::kZeros + j) = 0x08080808u;
    grid_dep_wait();
    grid_dep_launch();

    // The copies of a stage (steps s .. s + SPS - 1, as far as they belong to
    // this slice): 512 bytes a tile of words; scales (2 pieces of 16 bytes a
    // tile) and zero points (1 piece), a group each; and this warp's part of
    // the rows of x.  k_in ends on half a step if it is no multiple of 128.
    // Every lane's sources advance by the same distance from stage to stage.
    const int kt_end = min(2 * s1, kt_all);
    const uint4* words[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
        words[c] = reinterpret_cast<const uint4*>(p.packed) + ((long long)min(tn0 + c, tn_all - 1) * kt_all + 2 * s0) * 32 + lane;
    constexpr int kPieces = 3 * CT, kGroupPieces = SPS * kParts * kPieces, kMine = (kGroupPieces + 31) / 32;
    const unsigned char* piece[kMine];
    uint32_t piece_to[kMine];
    int piece_step[kMine], piece_group[kMine];               // group: past every k_in where there is none
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int i = lane + 32 * j, part = i / kPieces, r = i % kPieces;
        const long long at = (long long)(s0 * kParts + part) * p.n_out + 16 * tn0;
        const bool is_zero = r >= 2 * CT;
        piece[j] = is_zero ? p.zero + at + 16 * (r - 2 * CT) : reinterpret_cast<const unsigned char*>(p.scale + at + 8 * r);
        piece_to[j] = is_zero ? S::kZeros + part * (CT * 16) + (r - 2 * CT) * 16 : S::kScales + part * (CT * 32) + r * 16;
        piece_step[j] = SPS * kParts * p.n_out * (is_zero ? 1 : 2);
        piece_group[j] = i < kGroupPieces && (is_zero ? p.zero && r - 2 * CT < tiles : r < 2 * tiles) ? s0 * kParts + part : 1 << 30;
    }
    const int group_end = min(s1 * kParts, p.k_in / GROUP);
    // x: kCols threads along the inputs, the others of the warps that share it along the rows
    constexpr int kXPieces = SPS * 16;                       // of a row
    const int x_threads = 32 * p.warps_c, x_lane = wc * 32 + lane;
    const int x_cols = min(x_threads, kXPieces), x_rows = x_threads / x_cols, x_row = x_lane / x_cols, x_col = x_lane % x_cols;
    const uint16_t* x_from = p.x + (long long)x_row * p.k_in + 128 * s0 + 8 * x_col;
    const uint32_t x_to = smem_u32(x_ring) + x_row * S::kXRow + 16 * x_col;
    const long long x_next = (long long)x_rows * p.k_in;
    int fetched = s0;                                        // steps
    uint32_t* status = reinterpret_cast<uint32_t*>(p.ws);
    const long long scales_all = (long long)(p.k_in / GROUP) * p.n_out;          // and zero points
    auto fetch = [&](int stage) {
        const uint32_t to = smem_u32(ring) + stage * S::kStage;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
#pragma unroll
            for (int i = 0; i < 2 * SPS; ++i)
                if (2 * fetched + i < kt_end &&
                    guard(words[c] + i * 32 - reinterpret_cast<const uint4*>(p.packed) < (long long)tn_all * kt_all * 32, status))
                    copy16(to + c * (SPS * 1024) + i * 512 + lane * 16, words[c] + i * 32);
            words[c] += SPS * 64;
        }
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            if (piece_group[j] < group_end &&
                guard(piece_step[j] == SPS * kParts * p.n_out ? piece[j] - p.zero + 16 <= scales_all
                                                              : piece[j] - reinterpret_cast<const unsigned char*>(p.scale) + 16 <= 2 * scales_all, status))
                copy16(to + piece_to[j], piece[j]);
            piece[j] += piece_step[j];
            piece_group[j] += SPS * kParts;
        }
        const uint32_t xt = x_to + stage * p.m * S::kXRow;
        for (int col = 0; col < kXPieces; col += x_cols) {
            if (128 * fetched + 8 * (x_col + col) >= 64 * kt_end) break;
            const uint16_t* src = x_from + 8 * col;
            uint32_t dst = xt + 16 * col;
            for (int row = x_row; row < p.m; row += x_rows, src += x_next, dst += x_rows * S::kXRow)
                if (guard(src - p.x + 8 <= (long long)p.m * p.k_in, status)) copy16(dst, src);
        }
        x_from += SPS * 128;
        fetched += SPS;
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    for (int i = 0; i < depth - 1; ++i) {
        if (fetched < s1) fetch(i);
        commit();
    }

    float acc[CT][NT][4];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][n][e] = 0.f;
    // columns past the last row repeat it; their sums are not written
    int row_at[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) row_at[n] = min(8 * n + g, p.m - 1) * S::kXRow + 16 * t;

    float sum[CT][NT][4];
    __half2 zlo[CT], zhi[CT];
    // 64 inputs (the first or second tile of a step) from shared memory
    auto tile = [&](auto second, uint32_t words_at, const uint32_t (&x_at)[NT], uint32_t scales, uint32_t zeros) {
        constexpr int kSecond = decltype(second)::value;
        uint4 w[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) w[c] = lds16(words_at + c * (SPS * 1024) + kSecond * 512);
#pragma unroll
        for (int half = 0; half < 2; ++half) {               // 32 inputs
            const int k = 64 * kSecond + 32 * half, part = k / GROUP;
            const bool opens = k % GROUP == 0, closes = (k + 32) % GROUP == 0;
            if (opens) {
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const int ch = (part * CT + c) * 16;
                    // -(1024 + z) is the bits of -1024 with z in the last places; -(64 + z) is 960 more
                    zlo[c] = bits_h2(0xE400E400u | lds_byte(zeros + ch) * 0x10001u);
                    zhi[c] = __hadd2(bits_h2(0xE400E400u | lds_byte(zeros + ch + 8) * 0x10001u), __float2half2_rn(960.f));
                }
            }
            uint4 x[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n] = lds16(x_at[n] + 128 * kSecond + 64 * half);
#pragma unroll
            for (int i = 0; i < 2; ++i) {                    // k-steps of 16 inputs
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    uint32_t a[4];
                    q4_fragment(half ? (i ? w[c].w : w[c].z) : (i ? w[c].y : w[c].x), zlo[c], zhi[c], a);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint32_t b0 = i ? x[n].z : x[n].x, b1 = i ? x[n].w : x[n].y;
                        if (opens && i == 0) mma_16816_first(sum[c][n], a, b0, b1);
                        else mma_16816(sum[c][n], a, b0, b1);
                    }
                }
            }
            if (closes) {
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const int ch = (part * CT + c) * 16;
                    const float s_lo = lds_half(scales + 2 * ch), s_hi = lds_half(scales + 2 * ch + 16);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[c][n][e] += (e < 2 ? s_lo : s_hi) * sum[c][n][e];
                }
            }
        }
    };

    int stage = 0;
    for (int s = s0; s < s1; s += SPS) {
        // this stage has landed, for every warp that shares its rows, and the
        // one before it is read
        cp_async_wait(depth - 2);
        if (p.warps_c == 1) __syncwarp();
        else named_bar(1 + wk, x_threads);
        if (fetched < s1) fetch(stage == 0 ? depth - 1 : stage - 1);
        commit();
        const uint32_t at = smem_u32(ring) + stage * S::kStage;
        uint32_t words_at = at + lane * 16, scales = at + S::kScales + 2 * g, zeros = at + S::kZeros + g, x_at[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) x_at[n] = smem_u32(x_ring) + stage * p.m * S::kXRow + row_at[n];
        const int here = min(SPS, s1 - s);
#pragma unroll 1
        for (int i = 0; i < here; ++i) {
            tile(std::integral_constant<int, 0>{}, words_at, x_at, scales, zeros);
            if (2 * (s + i) + 1 < kt_all) tile(std::integral_constant<int, 1>{}, words_at, x_at, scales, zeros);
            words_at += 1024;
            scales += kParts * CT * 32;
            zeros += kParts * CT * 16;
#pragma unroll
            for (int n = 0; n < NT; ++n) x_at[n] += 256;
        }
        if (++stage == depth) stage = 0;
    }

    // join the warps along the inputs: red[wk][row][channel]
    const int ch_cta = 16 * CT * p.warps_c;
    __syncthreads();                                         // the rings are read
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 8 * n + 2 * t + (e & 1), ch = 16 * (CT * wc + c) + g + 8 * (e >> 1);
                red[(wk * S::kRows + row) * ch_cta + ch] = acc[c][n][e];
            }
    __syncthreads();
    const int row_vecs = ch_cta / 4, vecs = p.m * row_vecs;  // four channels at a time
    float4* red4 = reinterpret_cast<float4*>(smem);
    float4* part4 = reinterpret_cast<float4*>(p.ws + ws_data_off()) + (size_t)blockIdx.x * p.splits * vecs;
    for (int i = threadIdx.x; i < vecs; i += S::kThreads) {
        float4 s = red4[i];
        for (int v = 1; v < warps_k; ++v) {
            const float4 o = red4[v * (S::kRows * row_vecs) + i];
            s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
        }
        if (p.splits == 1) red4[i] = s;
        else if (guard(((long long)blockIdx.x * p.splits + blockIdx.y) * vecs + i < p.part_vecs, status))
            __stcg(part4 + (size_t)blockIdx.y * vecs + i, s);
    }
    if (p.splits > 1) {
        __threadfence();
        __syncthreads();
        uint32_t* counter = reinterpret_cast<uint32_t*>(p.ws + ws_counter_off()) + blockIdx.x;
        if (threadIdx.x == 0) {
            last_flag = atomicAdd(counter, 1u) == (uint32_t)p.splits - 1;
            if (last_flag) *counter = 0;
        }
        __syncthreads();
        if (!last_flag) return;
        __threadfence();
    }
    const int ch_here = min(ch_cta, p.n_out - (int)blockIdx.x * ch_cta);
    for (int i = threadIdx.x; i < vecs; i += S::kThreads) {
        const int row = i / row_vecs, ch = 4 * (i % row_vecs);
        if (ch >= ch_here) continue;
        float4 s;
        if (p.splits > 1) {
            s = __ldcg(part4 + i);
#pragma unroll 4
            for (int v = 1; v < p.splits; ++v) {
                const float4 o = __ldcg(part4 + (size_t)v * vecs + i);
                s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
            }
        } else {
            s = red4[i];                                     // written by this thread
        }
        const long long out = (long long)row * p.n_out + (long long)blockIdx.x * ch_cta + ch;
        if (!guard(out + 4 <= (long long)p.m * p.n_out, status)) continue;
        if (p.y_fp32) {
            *reinterpret_cast<float4*>(static_cast<float*>(p.y) + out) = s;
        } else {
            const __half2 lo = __floats2half2_rn(s.x, s.y), hi = __floats2half2_rn(s.z, s.w);
            *reinterpret_cast<uint2*>(static_cast<__half*>(p.y) + out) = make_uint2(h2_bits(lo), h2_bits(hi));
        }
    }
}

__global__ void __launch_bounds__(256) q4_pack_kernel(const uint8_t* __restrict__ q, int k_in, int n_out,
                                                      uint32_t* __restrict__ packed)
{
    grid_dep_wait();
    const long long words = (long long)k_in * n_out / 8;
    const int kt_all = k_in / 64;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += (long long)gridDim.x * blockDim.x) {
        const int j = (int)(i & 3), lane = (int)(i >> 2) & 31;
        const long long tile = i >> 7;
        const long long tn = tile / kt_all, tk = tile % kt_all;
        const long long k0 = 64 * tk + 32 * (j >> 1) + 8 * (lane & 3) + 4 * (j & 1), n0 = 16 * tn + (lane >> 2);
        uint32_t w = 0;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w |= (uint32_t)(q[(k0 + e) * n_out + n0 + 8 * c] & 15) << (4 * c + 8 * (e >> 1) + 16 * (e & 1));
        packed[i] = w;
    }
}

// How a product is cut.  Warps stream; what they have to be is many and long:
// the channel tiles of all warps times the cuts of the inputs should fill the
// GPU about once.  The cuts are first the warps of a CTA (joined in shared
// memory), then CTAs.  With more rows, warps of a CTA rather lie along the
// channels, so that x is read less often: a CTA then takes 8 m channels and
// more, and x is at most half the bytes of the weights.
struct Q4Plan {
    int shape, ct, warps_c, blocks, splits;
};

constexpr int most_rows(int shape) { return shape == 0 ? 2 : 8 * shape; }
constexpr int least_warps_c(int shape) { return shape == 0 ? 1 : shape == 1 ? 2 : 4; }

// Whether the other kernel takes the product.  It decodes faster and needs no
// more for 32 rows than for 9, but takes a launch more, 16 rows at least, and
// has a sum per group to read and scale.  This kernel against it, groups of 128:
// 8 rows of 5120 x 5120 8.4 and 9.4 us, 12 rows 10.8 and 9.4, 32 rows 17.0 and
// 10.3; 12 rows of 2048 x 2048 6.8 and 6.5.  Groups of 32: 16 rows of 17408 x
// 5120 22.5 and 26.2 us, 24 rows 27.7 and 31.6, 32 rows 36.3 and 31.7 (of small
// matrices the other is ahead earlier: 24 rows of 2048 x 2048 8.9 and 7.7).
bool takes_tc(int m, int group) { return m > (group == 32 ? 24 : 8); }

Q4Plan q4_plan(int m, int k_in, int n_out)
{
    Q4Plan pl;
    // Up to 2 rows warps of 16 channels have the deeper stages, and pay where a CTA
    // per 16 channels, whose warps split the inputs, finds a place at once: one row
    // of 4096 x 4096 4.3 us, warps of 32 channels 6.5; of 17408 x 5120 19.9, 16.0.
    pl.shape = m <= 2 && n_out / 16 <= 148 * 2 ? 0 : m <= 8 ? 1 : m <= 16 ? 2 : 3;
    pl.ct = pl.shape == 0 ? 1 : 2;
    const int steps = (k_in / 64 + 1) / 2, tiles = (n_out / 16 + pl.ct - 1) / pl.ct;
    const int warps = 148 * 8 * 2;
    int cuts = warps / tiles;                                // of the inputs
    if (cuts > steps / 2) cuts = steps / 2;
    if (cuts < 1) cuts = 1;
    pl.warps_c = 8;
    while (pl.warps_c > least_warps_c(pl.shape) && 16 / pl.warps_c <= cuts) pl.warps_c /= 2;
    pl.blocks = (tiles + pl.warps_c - 1) / pl.warps_c;
    pl.splits = cuts / (8 / pl.warps_c);
    if (pl.splits < 1 || pl.blocks > kMaxBlocks) pl.splits = 1;
    return pl;
}

template <int SHAPE, int CT, int NT, int SPS, int GROUP>
cudaError_t launch_q4_t(Q4Args a, const Q4Plan& pl, cudaStream_t stream)
{
    using S = Q4Shape<CT, NT, SPS, GROUP>;
    auto kern = q4_gemm_kernel<CT, NT, SPS, GROUP>;
    // as many stages as fit beside kMinCtas - 1 other CTAs on an SM, whose 228 KB hold 1 KB of the system's a CTA;
    // two at least, whatever the rows and the cut
    const int stage = S::kWarps * S::kStage + S::kWarps / pl.warps_c * a.m * S::kXRow;
    constexpr int kRoom = 227 * 1024 / S::kMinCtas - 1024;
    static_assert(2 * (S::kWarps * S::kStage + S::kWarps / least_warps_c(SHAPE) * most_rows(SHAPE) * S::kXRow) <= kRoom,
                  "a ring needs two stages");
    a.depth = kRoom / stage;
    if (a.depth > kQ4MaxDepth) a.depth = kQ4MaxDepth;
    const int join = (int)sizeof(float) * S::kWarps * 16 * CT * S::kRows;
    const int smem = a.depth * stage > join ? a.depth * stage : join;
    static std::atomic<int> done[kMaxDevices];
    const cudaError_t e = once_per_device(done, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)pl.blocks, (unsigned)pl.splits), dim3(S::kThreads), (size_t)smem, stream, a);
}

template <int SHAPE, int CT, int NT, int SPS>
cudaError_t launch_q4_g(const Q4Args& a, const Q4Plan& pl, int group, cudaStream_t stream)
{
    return group == 32 ? launch_q4_t<SHAPE, CT, NT, SPS, 32>(a, pl, stream)
                       : group == 64 ? launch_q4_t<SHAPE, CT, NT, SPS, 64>(a, pl, stream) : launch_q4_t<SHAPE, CT, NT, SPS, 128>(a, pl, stream);
}

}  // namespace

size_t q4_workspace_need(int m, int k_in, int n_out, int group)
{
    if (takes_tc(m, group)) return q4_tc_workspace_bytes(m, k_in, n_out);
    const Q4Plan pl = q4_plan(m, k_in, n_out);
    return ws_data_off() + (pl.splits == 1 ? 0 : align_up(sizeof(float) * (size_t)pl.blocks * pl.splits * 16 * pl.ct * pl.warps_c * m, 256));
}

size_t q4_workspace_bytes(int m, int k_in, int n_out)
{
    size_t most = 0;
    for (int rows = 1; rows <= m; ++rows)
        for (int group = 32; group <= 64; group *= 2) {      // (128 as 64)
            const size_t need = q4_workspace_need(rows, k_in, n_out, group);
            if (need > most) most = need;
        }
    return most;
}

cudaError_t launch_q4_gemm(int m, const uint16_t* x, const uint32_t* packed, const uint16_t* scale,
                           const uint8_t* zero, void* y, int y_fp32, int k_in, int n_out, int group,
                           unsigned char* ws, cudaStream_t stream)
{
    if (takes_tc(m, group)) return launch_q4_tc(m, x, packed, scale, zero, y, y_fp32, k_in, n_out, group, ws, stream);
    const Q4Plan pl = q4_plan(m, k_in, n_out);
    const Q4Args a = {x, packed, scale, zero, y, m, k_in, n_out, y_fp32 ? 1 : 0, pl.warps_c, pl.splits, 0, ws,
                      (long long)(q4_workspace_need(m, k_in, n_out, group) - ws_data_off()) / 16};
    switch (pl.shape) {
        case 0: return launch_q4_g<0, 1, 1, 4>(a, pl, group, stream);
        case 1: return launch_q4_g<1, 2, 1, 2>(a, pl, group, stream);
        case 2: return launch_q4_t<2, 2, 2, 2, 32>(a, pl, stream);
        default: return launch_q4_t<3, 2, 3, 1, 32>(a, pl, stream);
    }
}

cudaError_t launch_q4_pack(const uint8_t* q, int k_in, int n_out, uint32_t* packed, cudaStream_t stream)
{
    const long long words = (long long)k_in * n_out / 8;
    const long long blocks = (words + 255) / 256;
    return launch_pdl(q4_pack_kernel, dim3((unsigned)(blocks < 148 * 16 ? blocks : 148 * 16)), dim3(256), 0, stream, q,
                      k_in, n_out, packed);
}

}  // namespace exl3
