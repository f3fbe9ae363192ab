// q4.cu -- products with plain 4-bit weights in groups (exl3_q4_gemm), and
// their packing.
//
//     y[i][n] = sum_k x[i][k] (q[k][n] - z[k/g][n]) s[k/g][n],   1..32 rows
//
// The product reads half a byte per weight and does 2 m flops with it, so at
// few rows the stream of packed words is the bound.  What a weight may cost
// in instructions at that rate is about three; the kernel spends a little
// over one:
//   * The packed tiles (16 channels x 64 inputs, layout in include/exl3.h) are
//     the A operand of mma.m16n8k16 in register order: a lane's 128-bit load
//     is its share of four k-steps.  Two fields of a word become an fp16 pair
//     by one OR into the mantissa of 1024 (fields at bits 0 and 16) or of
//     1024 again with the field worth 16 (bits 4 and 20), and one packed add
//     or FMA takes the bias and the zero point off.  Both are exact: |q - z|
//     is an integer below 2048, for any uint8 zero.
//   * x is the B operand straight from global memory (the few rows live in
//     L1): a lane reads 8 consecutive inputs of its row per 32-input block.
//   * The fp32 sums of a group are scaled in fp32 and added up; nothing is
//     rounded below 32 bits before the result.
// A warp takes a run of 64-input tiles of 16*CT channels; the warps of a CTA
// and the CTAs of a cut (grid.y) split the inputs.  Sums are joined in warp
// order in shared memory, and in CTA order by the last CTA to arrive.
#include <cuda_fp16.h>

#include "exl3_common.cuh"
#include "exl3_internal.h"

namespace exl3 {

namespace {

constexpr int kQ4Warps = 8;
constexpr int kQ4Threads = 32 * kQ4Warps;

struct Q4Args {
    const uint16_t* x;
    const uint32_t* packed;
    const uint16_t* scale;
    const uint8_t* zero;
    void* y;
    int m, k_in, n_out, y_fp32;
    int splits;               // CTAs that share a channel block's inputs
    unsigned char* ws;
};

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The A fragment of one k-step: rows g (lo) and g + 8 (hi) of the tile.
// zlo = -(1024 + z) and zhi = -(64 + z) as pairs.
__device__ __forceinline__ void q4_fragment(uint32_t w, __half2 zlo, __half2 zhi, uint32_t (&a)[4])
{
    const __half2 sixteenth = __float2half2_rn(0.0625f);
    const uint32_t v = w >> 8;
    a[0] = h2_bits(__hadd2(bits_h2((w & 0x000F000Fu) | 0x64006400u), zlo));
    a[1] = h2_bits(__hfma2(bits_h2((w & 0x00F000F0u) | 0x64006400u), sixteenth, zhi));
    a[2] = h2_bits(__hadd2(bits_h2((v & 0x000F000Fu) | 0x64006400u), zlo));
    a[3] = h2_bits(__hfma2(bits_h2((v & 0x00F000F0u) | 0x64006400u), sixteenth, zhi));
}

template <int CT, int NT, int GROUP>
__global__ void __launch_bounds__(kQ4Threads) q4_gemm_kernel(Q4Args p)
{
    constexpr int kBlockCh = 16 * CT;
    constexpr int kRows = 8 * NT;
    extern __shared__ __align__(16) float red[];            // warps x channels x rows
    __shared__ int last_flag;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int kt_all = p.k_in / 64;
    const int tn0 = blockIdx.x * CT, tn_all = p.n_out / 16;
    const int slice = blockIdx.y * kQ4Warps + warp, slices = p.splits * kQ4Warps;
    const int kt0 = (int)((long long)kt_all * slice / slices), kt1 = (int)((long long)kt_all * (slice + 1) / slices);

    grid_dep_wait();
    grid_dep_launch();

    float acc[CT][NT][4];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][n][e] = 0.f;

    for (int kt = kt0; kt < kt1; ++kt) {
        uint4 w[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int tn = min(tn0 + c, tn_all - 1);
            w[c] = __ldg(reinterpret_cast<const uint4*>(p.packed) + ((long long)tn * kt_all + kt) * 32 + lane);
        }
        uint4 b[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = 8 * n + g;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                b[n][h] = row < p.m ? *reinterpret_cast<const uint4*>(p.x + (long long)row * p.k_in + 64 * kt + 32 * h + 8 * t)
                                    : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int ch = 16 * min(tn0 + c, tn_all - 1) + g;
            const uint32_t words[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
            constexpr int kParts = GROUP == 32 ? 2 : 1;      // groups inside the 64 inputs
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                const long long at = (long long)((64 * kt) / GROUP + part) * p.n_out + ch;
                const float s_lo = __half2float(__ushort_as_half(p.scale[at]));
                const float s_hi = __half2float(__ushort_as_half(p.scale[at + 8]));
                const int z_lo = p.zero ? p.zero[at] : 8, z_hi = p.zero ? p.zero[at + 8] : 8;
                const __half2 zlo = __half2half2(__int2half_rn(-1024 - z_lo)), zhi = __half2half2(__int2half_rn(-64 - z_hi));
                float sum[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[n][e] = 0.f;
#pragma unroll
                for (int j = part * (4 / kParts); j < (part + 1) * (4 / kParts); ++j) {
                    uint32_t a[4];
                    q4_fragment(words[j], zlo, zhi, a);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 bb = b[n][j >> 1];
                        if (j & 1) mma_16816(sum[n], a, bb.z, bb.w);
                        else mma_16816(sum[n], a, bb.x, bb.y);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[c][n][0] += s_lo * sum[n][0];
                    acc[c][n][1] += s_lo * sum[n][1];
                    acc[c][n][2] += s_hi * sum[n][2];
                    acc[c][n][3] += s_hi * sum[n][3];
                }
            }
        }
    }

    // join the warps: red[warp][row][channel]
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 8 * n + 2 * t + (e & 1), ch = 16 * c + g + 8 * (e >> 1);
                red[(warp * kRows + row) * kBlockCh + ch] = acc[c][n][e];
            }
    __syncthreads();
    const int ch_here = min(kBlockCh, p.n_out - tn0 * 16);
    float* part = reinterpret_cast<float*>(p.ws + ws_data_off()) +
                  (size_t)(blockIdx.x * p.splits) * (kBlockCh * p.m);
    for (int i = threadIdx.x; i < p.m * kBlockCh; i += kQ4Threads) {
        float s = red[i];
#pragma unroll
        for (int v = 1; v < kQ4Warps; ++v) s += red[v * kRows * kBlockCh + i];
        red[i] = s;
        if (p.splits > 1) part[(size_t)blockIdx.y * (kBlockCh * p.m) + i] = s;
    }
    if (p.splits > 1) {
        __threadfence();
        __syncthreads();
        uint32_t* counter = reinterpret_cast<uint32_t*>(p.ws + ws_counter_off()) + blockIdx.x;
        if (threadIdx.x == 0) last_flag = atomicAdd(counter, 1u) == (uint32_t)p.splits - 1;
        __syncthreads();
        if (!last_flag) return;
        if (threadIdx.x == 0) *counter = 0;
        __threadfence();
        for (int i = threadIdx.x; i < p.m * kBlockCh; i += kQ4Threads) {
            float s = 0.f;
            for (int v = 0; v < p.splits; ++v) s += __ldcg(part + (size_t)v * (kBlockCh * p.m) + i);
            red[i] = s;
        }
    }
    // every thread reads back what it wrote itself: no barrier is needed
    for (int i = threadIdx.x; i < p.m * kBlockCh; i += kQ4Threads) {
        const int row = i / kBlockCh, ch = i % kBlockCh;
        if (ch >= ch_here) continue;
        const long long at = (long long)row * p.n_out + tn0 * 16 + ch;
        if (p.y_fp32) static_cast<float*>(p.y)[at] = red[i];
        else static_cast<__half*>(p.y)[at] = __float2half_rn(red[i]);
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

struct Q4Plan {
    int ct, nt, blocks, splits;
};

Q4Plan q4_plan(int m, int k_in, int n_out)
{
    Q4Plan pl;
    pl.nt = m <= 8 ? 1 : m <= 16 ? 2 : 4;
    pl.ct = pl.nt;
    pl.blocks = (n_out / 16 + pl.ct - 1) / pl.ct;
    const int slots = 148 * (pl.nt == 1 ? 4 : 2);
    int s = slots / pl.blocks;
    const int most = (k_in / 64 + 2 * kQ4Warps - 1) / (2 * kQ4Warps);
    if (s > most) s = most;
    if (s < 1 || pl.blocks > kMaxBlocks) s = 1;
    pl.splits = s;
    return pl;
}

template <int CT, int NT>
cudaError_t launch_q4_t(const Q4Args& a, const Q4Plan& pl, int group, cudaStream_t stream)
{
    auto kern = group == 32 ? q4_gemm_kernel<CT, NT, 32>
                            : group == 64 ? q4_gemm_kernel<CT, NT, 64> : q4_gemm_kernel<CT, NT, 128>;
    constexpr size_t smem = sizeof(float) * kQ4Warps * 16 * CT * 8 * NT;
    if (smem > 48 * 1024) {
        static std::atomic<int> done[3][kMaxDevices];
        cudaError_t e = once_per_device(done[group == 32 ? 0 : group == 64 ? 1 : 2], [&] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        });
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kern, dim3((unsigned)pl.blocks, (unsigned)pl.splits), dim3(kQ4Threads), smem, stream, a);
}

}  // namespace

size_t q4_workspace_bytes(int m, int k_in, int n_out)
{
    const Q4Plan pl = q4_plan(m, k_in, n_out);
    if (pl.splits == 1) return ws_data_off();
    return ws_data_off() + align_up(sizeof(float) * (size_t)pl.blocks * pl.splits * 16 * pl.ct * m, 256);
}

cudaError_t launch_q4_gemm(int m, const uint16_t* x, const uint32_t* packed, const uint16_t* scale,
                           const uint8_t* zero, void* y, int y_fp32, int k_in, int n_out, int group,
                           unsigned char* ws, cudaStream_t stream)
{
    const Q4Plan pl = q4_plan(m, k_in, n_out);
    const Q4Args a = {x, packed, scale, zero, y, m, k_in, n_out, y_fp32 ? 1 : 0, pl.splits, ws};
    switch (pl.nt) {
        case 1: return launch_q4_t<1, 1>(a, pl, group, stream);
        case 2: return launch_q4_t<2, 2>(a, pl, group, stream);
        default: return launch_q4_t<4, 4>(a, pl, group, stream);
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
