// q4_tc.cu -- products with plain 4-bit weights in groups (exl3_q4_gemm) of more
// than 8 rows (24 in groups of 32), on the fifth-generation tensor cores.
//
//     y[i][n] = sum_k x[i][k] (q[k][n] - z[k/g][n]) s[k/g][n]
//
// A CTA takes 128 output channels, the M side of tcgen05.mma, and the rows of
// x, up to 32, as its N side; inputs come in stages of 128.
//   * The weights are the A operand in tensor memory.  A lane's word of the
//     packed layout (channels g and g + 8, four inputs each) becomes four
//     registers, one AND-OR and one packed add each: (q - z) as an exact fp16
//     integer.  That is the register layout of tcgen05.st.16x256b: a tile of 16
//     channels x 64 inputs, a 128-bit read a lane, is one store instruction.
//     Nothing goes back through shared memory, whose bandwidth would be the
//     bound (32 KB written and read again a stage); the store takes 130 clocks
//     a stage, the eight MMAs 128 (32 rows) or 73 (16), of the 350 that the
//     memory gives.
//   * The order of inputs in an MMA's K is the packed layout's: 16 of 32 inputs,
//     those of the words 2 j or 2 j + 1.  x is brought into shared memory in
//     that order, in pieces of four inputs (8 bytes).
//     A small kernel in front lays it out so, once for all CTAs, and a bulk copy
//     brings a stage.  (Copies of 8 bytes by every CTA for itself kept four warps
//     busy, 32 requests a stage.)
//   * Each group of inputs has its own sum in tensor memory.  Scaler warps read
//     it, a channel a thread, scale it in fp32 and add it up.  Nothing is rounded
//     below 32 bits before the result.
// What bounds it is the issue of instructions (1700 a stage, most of them the
// decoders'), 0.38 us a stage and CTA where memory would give 0.18; below that,
// about 5 us for the launches, the first bytes and the end.  Two sets of warps
// take stages in turn, so that one stage's waits are another's work: a wait on a
// barrier costs 150 clocks even if its phase is over.  32 rows of 5120 x 17408 in
// groups of 128 take 18.5 us (2.6 TB/s; on the legacy tensor pipe 29.3), 16 rows
// 16.9 (19.6), 32 rows of 5120 x 5120 10.3 (17.0).
// CTAs that split the inputs of a block of channels are a cluster; they add up
// their parts, in order, through each other's shared memory (through memory and
// the last one to arrive: 15.0 us for 5120 x 5120).
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "exl3_cache.h"
#include "exl3_pipe.cuh"
#include "exl3_tc.cuh"

namespace exl3 {

namespace {

namespace cg = cooperative_groups;

struct Q4TcArgs {
    const uint16_t* x;
    const uint32_t* packed;
    const uint16_t* scale;
    const uint8_t* zero;
    void* y;
    int m, k_in, n_out, y_fp32;
    int splits;
    unsigned char* ws;
    const unsigned char* xt;  // x as the stages want it, in the workspace
    size_t xt_bytes;
};

// Warps: two sets of eight decoders, of four scalers and of one that issues MMAs
// take stages in turn; one brings x.
constexpr int kSets = 2, kDecoders = 8, kScalers = 4;        // of a set
constexpr int kFirstScaler = kSets * kDecoders, kBringer = kFirstScaler + kSets * kScalers, kFirstIssuer = kBringer + 1;
constexpr int kTcThreads = 32 * (kFirstIssuer + kSets);
constexpr int kScaleRing = 16;                               // groups

template <int N>
constexpr int kXStage = 2 * N * 128;                         // bytes of x of a stage: two halves of 64 inputs, 128-byte swizzle

template <int N, int GROUP>
struct Q4Tc {
    static constexpr int kParts = 128 / GROUP;               // groups of a stage
    static constexpr int kRing = 8;                          // stages of x in shared memory
    static constexpr int kA = 4;                             // stages of weights in tensor memory
    static constexpr int kD = 8 / kParts;                    // stages whose groups' sums lie there
    static constexpr int kCols = 512;
    static constexpr int kSums = 64 * kA;                    // first column of the sums
    static_assert(kSums + kD * kParts * N <= kCols);
    static_assert(kRing % kA == 0 && kA % kSets == 0 && kRing % kD == 0 && kD % kSets == 0);
    static constexpr int kWords = 1024;                      // of a decoder's stage
    static constexpr int kOwnRing = 8;                       // stages of a decoder in shared memory
    static_assert(kSets == 2 && kRing == 8 && kA == 4 && kOwnRing == 8);         // the decoders' loop is written for it
    static constexpr int kXAll = kRing * kXStage<N>, kOwnAll = kOwnRing * kSets * kDecoders * kWords;
    static constexpr int kZeros = kSets * kDecoders * 1024;
    static constexpr int kScales = kSets * kScalers * kScaleRing * 64;
    static constexpr int kSmem = kXAll + kOwnAll + kZeros + kScales + 512;
    static_assert(kSmem <= 227 * 1024);
};

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// The pair's fields in the mantissa of 1024, in one instruction.
__device__ __forceinline__ __half2 masked_1024(uint32_t w, uint32_t mask)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(mask), "r"(0x64006400u));
    return bits_h2(r);
}

// A word as the fp16 pairs q - z of channel g (inputs 0 1, 2 3) and g + 8, from
// 1024 + q and 1024 + 16 q: zlo = -(1024 + z), zhi = -(64 + z).
__device__ __forceinline__ void decode_word(uint32_t w, __half2 zlo, __half2 zhi, uint32_t* a)
{
    const uint32_t v = w >> 8;
    const __half2 sixteenth = __float2half2_rn(0.0625f);
    a[0] = h2_bits(__hadd2(masked_1024(w, 0x000F000Fu), zlo));
    a[1] = h2_bits(__hadd2(masked_1024(v, 0x000F000Fu), zlo));
    a[2] = h2_bits(__hfma2(masked_1024(w, 0x00F000F0u), sixteenth, zhi));
    a[3] = h2_bits(__hfma2(masked_1024(v, 0x00F000F0u), sixteenth, zhi));
}

// 16 lanes x 32 columns of tensor memory: lane (g, t) of the warp holds columns
// 2 t and 2 t + 1 of each eight, of lane g (registers 0 1 of four) and g + 8.
__device__ __forceinline__ void tmem_st_tile(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D (+)= A B over 32 inputs, two MMAs with A in tensor memory, issued by one
// elected lane.
__device__ __forceinline__ void mma_f16_ts_pair_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %3, %5, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %4, %5, 1;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(a_tmem + 8), "l"(bdesc), "l"(bdesc + 2), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last GROUPS groups of this thread's copies have landed.
template <int GROUPS>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(GROUPS) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
// d += a b for two floats at once.
__device__ __forceinline__ void fma2(float2& d, float2 a, float2 b)
{
    uint64_t& dd = reinterpret_cast<uint64_t&>(d);
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(dd) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
}
__device__ __forceinline__ uint32_t lds_byte(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}

template <int N, int GROUP>
__global__ void __launch_bounds__(kTcThreads, 1) q4_tc_kernel(const __grid_constant__ Q4TcArgs p)
{
    using S = Q4Tc<N, GROUP>;
    constexpr int kParts = S::kParts;
    extern __shared__ __align__(1024) unsigned char smem[];  // the swizzle counts rows from 1024-byte borders
    unsigned char* own_all = smem + S::kXAll;
    unsigned char* zero_all = own_all + S::kOwnAll;
    unsigned char* scales = zero_all + S::kZeros;
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + S::kScales);
    uint64_t* done = full + S::kRing;                        // a stage's weights and x are there; its MMAs are done
    uint64_t* read = done + S::kRing;                        // a stage's sums are read
    uint64_t* all_done = read + S::kD;
    uint32_t* tmem_base = reinterpret_cast<uint32_t*>(all_done + 1);
    static_assert((2 * S::kRing + S::kD + 1) * 8 + 4 <= 512);

    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
    const int kt_all = p.k_in / 64, stages = (kt_all + 1) / 2;
    const int s0 = (int)((long long)stages * blockIdx.x / p.splits), s1 = (int)((long long)stages * (blockIdx.x + 1) / p.splits);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kRing; ++i) {
            mbar_init(full + i, kDecoders + 1);
            mbar_init(done + i, 1);
        }
        for (int i = 0; i < S::kD; ++i) mbar_init(read + i, kScalers);
        mbar_init(all_done, kSets);
        fence_mbar_init();
    }
    // Only the warp that brings x waits for the kernel before: that one started its
    // own dependents behind its wait, so all that came before it is done (weights
    // may be read, and nothing that is still to run asks for tensor memory).
    grid_dep_launch();
    if (warp == kFirstIssuer) {
        tmem_alloc(tmem_base, S::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_base;
    uint32_t* status = reinterpret_cast<uint32_t*>(p.ws);
    Patience wait = {status, true};

    if (warp < kFirstScaler) {
        // ------------------------------------------------------ decoders ---
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");  // 16 warps give up 16 registers a thread, 8 take 32
        // Unrolled over four stages of the set, one round of the ring of stages: what
        // a stage costs beside its arithmetic is most of these warps' instructions.
        const int set = warp / kDecoders, quarter = warp & 3, half = (warp >> 2) & 1;   // of the 128 lanes; of a quarter's 32
        const int tn_all = p.n_out / 16, tn = min((int)blockIdx.y * 8 + 2 * quarter + half, tn_all - 1);
        const int first = s0 + set, s_whole = kt_all / 2;    // k_in may end on half a stage
        const uint32_t own = smem_u32(own_all) + warp * (S::kOwnRing * S::kWords) + lane * 16;
        const uint4* words = reinterpret_cast<const uint4*>(p.packed) + ((long long)tn * kt_all + 2 * first) * 32 + lane;
        auto fetch = [&](int stage, int ahead, uint32_t to) {      // `ahead`: of the set's stages, from words on
            const uint4* from = words + ahead * (64 * kSets);
            const auto in = [&](const uint4* w) {
                return guard(w - reinterpret_cast<const uint4*>(p.packed) < (long long)tn_all * kt_all * 32, status);
            };
            if (stage < s1 && in(from)) copy16(to, from);
            if (stage < s1 && stage < s_whole && in(from + 32)) copy16(to + 512, from + 32);
            copies_commit();
        };
        // Zero points: a copy of the warp brings 16 bytes of 32 groups, one such chunk ahead.
        const uint32_t zero_ring = smem_u32(zero_all) + warp * 1024;
        constexpr int kStagesOf32 = 32 / kParts;             // of the set, that have 32 groups
        int z_group = (first + kSets * (lane / kParts)) * kParts + lane % kParts;
        const int z_end = min(s1 * kParts, p.k_in / GROUP);
        const uint8_t* zeros = p.zero ? p.zero + (long long)z_group * p.n_out + 16 * tn : nullptr;
        auto fetch_zeros = [&](int chunk) {
            if (p.zero) {
                if (z_group < z_end && guard(zeros - p.zero + 16 <= (long long)(p.k_in / GROUP) * p.n_out, status))
                    copy16(zero_ring + (chunk & 1) * 512 + 16 * lane, zeros);
                z_group += 32 * kSets;
                zeros += (long long)(32 * kSets) * p.n_out;
            }
        };
        if (!p.zero)
            for (int i = 0; i < 8; ++i) asm volatile("st.shared.u32 [%0], %1;" ::"r"(zero_ring + 128 * i + 4 * lane), "r"(0x08080808u) : "memory");
        fetch_zeros(0);
        fetch_zeros(1);
        for (int i = 0; i < S::kOwnRing - 1; ++i) fetch(first + kSets * i, i, own + i * S::kWords);
        words += (S::kOwnRing - 1) * 64 * kSets;
        const uint32_t to0 = tmem + ((uint32_t)(32 * quarter + 16 * half) << 16) + 64 * set;
        uint32_t z_at = lane >> 2;
        int n = 0;                                           // of the set's stages
        for (int s = first; s < s1; n += 4, words += 4 * 64 * kSets) {
            const uint32_t now = own + (n & 4) * S::kWords, then = own + (~n & 4) * S::kWords;
#pragma unroll
            for (int j = 0; j < 4; ++j, s += kSets) {
                if (s >= s1) break;
                copies_wait<S::kOwnRing - 2>();
                __syncwarp();
                // to the places of the stage, and of the zero points, before
                if (j == 0 && n > 0 && n % kStagesOf32 == 0) fetch_zeros(n / kStagesOf32 + 1);
                fetch(s + kSets * (S::kOwnRing - 1), j, (j ? now : then) + (j + 3) % 4 * S::kWords);
                // the MMAs of the stage whose weights lay where this one's will: four stages ago
                wait.wait(done + set + (2 * j + S::kRing - S::kA) % S::kRing, (n / 4 + (j < 2)) & 1);
                tc_fence_after();
                __half2 zlo, zhi;
#pragma unroll
                for (int tile = 0; tile < 2; ++tile) {
                    if (tile == 1 && s >= s_whole) break;
                    const uint4 w4 = lds16(now + j * S::kWords + 512 * tile);
                    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
                    uint32_t r[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = 64 * tile + 32 * (i >> 1);
                        if (i % 2 == 0 && k % GROUP == 0) {
                            // -(1024 + z) is the bits of -1024 with z in the last places; -(64 + z) is 960 more
                            const uint32_t z = zero_ring + z_at + 16 * (kParts * j + k / GROUP);
                            zlo = bits_h2(0xE400E400u | lds_byte(z) * 0x10001u);
                            zhi = __hadd2(bits_h2(0xE400E400u | lds_byte(z + 8) * 0x10001u), __float2half2_rn(960.f));
                        }
                        decode_word(w[i], zlo, zhi, r + 4 * i);
                    }
                    tmem_st_tile(to0 + 128 * (j & 1) + 32 * tile, r);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + set + 2 * j);
            }
            z_at = (z_at + 64 * kParts) % 1024;
        }
        copies_wait<0>();
    } else if (warp == kBringer) {
        // ------------------------------------------------------------- x ---
        grid_dep_wait();                                     // the kernel before lays x out
        // a nonzero injection word, low byte v (tests of the timeout path), lets the first v - 1 copies through
        const uint32_t inject = *reinterpret_cast<const volatile uint32_t*>(p.ws + kWsInjectOff);
        const int most = inject ? max((int)(inject & 255u) - 1, 0) : 0x7fffffff;
        Turn<S::kRing> slot;
        int issued = 0;
        for (int s = s0; s < s1 && issued < most; ++s, ++issued) {
            wait.wait(done + slot.at, slot.phase ^ 1);
            if (!wait.alive || !guard((size_t)(s + 1) * kXStage<N> <= p.xt_bytes, status)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(full + slot.at, kXStage<N>);
                bulk_g2s(smem + slot.at * kXStage<N>, p.xt + (size_t)s * kXStage<N>, kXStage<N>, full + slot.at);
            }
            __syncwarp();
            slot.next();
        }
        copies_landed<S::kRing>(full, issued, wait.status);
    } else if (warp < kBringer) {
        // ------------------------------------------------------- scalers ---
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int set = (warp - kFirstScaler) / kScalers, quarter = warp & 3, ch0 = blockIdx.y * 128 + 32 * quarter, ch = ch0 + lane;
        const int first = s0 + set, groups = p.k_in / GROUP;
        // Scales: a copy of the warp brings the 64 bytes of eight groups, eight groups ahead.
        const uint32_t ring = smem_u32(scales) + (warp - kFirstScaler) * (kScaleRing * 64);
        constexpr int kStagesOf8 = 8 / kParts;               // that have eight groups
        const int f_part = (lane >> 2) % kParts;
        int f_stage = first + kSets * ((lane >> 2) / kParts);
        const uint16_t* from = p.scale + ((long long)f_stage * kParts + f_part) * p.n_out + ch0 + 8 * (lane & 3);
        const bool brings = ch0 + 8 * (lane & 3) < p.n_out;
        uint32_t f_at = 0;
        auto fetch = [&] {
            if (brings && f_stage < s1 && f_stage * kParts + f_part < groups &&
                guard(from - p.scale + 8 <= (long long)groups * p.n_out, status))
                copy16(ring + f_at + 16 * lane, from);
            copies_commit();
            from += (long long)(kSets * 8) * p.n_out;
            f_stage += kSets * kStagesOf8;
            f_at = (f_at + 512) % (kScaleRing * 64);
        };
        for (int i = 0; i < kScaleRing / 8 - 1; ++i) fetch();
        float2 acc[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) acc[i] = make_float2(0.f, 0.f);
        Turn<S::kRing> here;
        Turn<S::kD> d;
        here.at = d.at = set;
        uint32_t at = 2 * lane;
        for (int s = first; s < s1; s += kSets) {
            if (at % 512 < 64) {
                copies_wait<kScaleRing / 8 - 2>();
                __syncwarp();                                // every lane has read the eight before, whose place is the next copy's
                fetch();
            }
            float sc[kParts];
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                uint16_t sh;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(sh) : "r"(ring + at + 64 * part));
                sc[part] = __half2float(__ushort_as_half(sh));
            }
            wait.wait(done + here.at, here.phase);
            tc_fence_after();
            const uint32_t sums = tmem + ((uint32_t)(32 * quarter) << 16) + S::kSums + d.at * (kParts * N);
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                if (s * kParts + part >= groups) break;
#pragma unroll
                for (int c = 0; c < N; c += 16) {            // (all at once would take more registers than there are)
                    uint32_t r[16];
                    tmem_ld16(sums + part * N + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        fma2(acc[c / 2 + i], make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])),
                             make_float2(sc[part], sc[part]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(read + d.at);
            at = (at + 64 * kParts) % (kScaleRing * 64);
            here.template next<kSets>();
            d.template next<kSets>();
        }
        copies_wait<0>();
        // the sets' sums, through the ring of the second set's decoders, whose last stage is done
        float* mine = reinterpret_cast<float*>(own_all + S::kOwnAll / 2) + 32 * quarter + lane;
        static_assert(N * 128 * 4 <= S::kOwnAll / 2);
        if (set == 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) mine[i * 128] = i & 1 ? acc[i / 2].y : acc[i / 2].x;
        }
        named_bar(2, 32 * kSets * kScalers);
        if (set == 0) {
            float y[N];
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] = (i & 1 ? acc[i / 2].y : acc[i / 2].x) + mine[i * 128];
            // ---- the result, or a part of it ----
            if (p.splits > 1) {
                float* part = reinterpret_cast<float*>(own_all) + 32 * quarter + lane;       // where the first set's decoders had their ring
#pragma unroll
                for (int i = 0; i < N; ++i) part[i * 128] = y[i];
            } else if (ch < p.n_out) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (i < p.m && guard((long long)i * p.n_out + ch < (long long)p.m * p.n_out, status)) {
                        if (p.y_fp32) static_cast<float*>(p.y)[(long long)i * p.n_out + ch] = y[i];
                        else static_cast<__half*>(p.y)[(long long)i * p.n_out + ch] = __float2half_rn(y[i]);
                    }
            }
        }
    } else {
        // ----------------------------------------------------- MMA warps ---
        // Unrolled over the ring, so that addresses are a base and constants: what
        // one of these warps executes is the longest chain of a stage.
        constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);     // f32 += f16 x f16, both K-major
        const int set = warp - kFirstIssuer;
        const uint64_t x0 = sdesc_sw128(smem_u32(smem) + set * kXStage<N>, 16, 1024);
        const uint32_t a0 = tmem + 64 * set, d0 = tmem + S::kSums + set * (kParts * N);
        uint32_t round = 0;                                  // of the ring: its parity is the barriers' phase
        for (int base = s0 + set; base < s1 && wait.alive; base += S::kRing, ++round) {
#pragma unroll
            for (int i = 0; i < S::kRing; i += kSets) {
                if (base + i >= s1) break;
                const bool whole = 2 * (base + i) + 1 < kt_all;
                wait.wait(read + set + i % S::kD, (round * (S::kRing / S::kD) + i / S::kD + 1) & 1);
                wait.wait(full + set + i, round & 1);
                tc_fence_after();
                if (!wait.alive) break;
#pragma unroll
                for (int k = 0; k < 128; k += 32)
                    if (k < 64 || whole)
                        mma_f16_ts_pair_elect(d0 + (i % S::kD * kParts + k / GROUP) * N, a0 + 64 * (i % S::kA) + k / 2,
                                              x0 + (i * kXStage<N> + (k >> 6) * (N * 128) + 2 * (k & 63)) / 16, idesc, k % GROUP != 0);
                mma_commit_elect(done + set + i);
            }
        }
        mma_commit_elect(all_done);                          // before tensor memory is given back
        (void)mbar_wait_bounded(all_done, 0, 100000000ull);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kFirstIssuer) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kCols);
    }
    if (p.splits > 1) {
        // the parts of the inputs, in order; each CTA of the cluster adds up some of the rows
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        float* part = reinterpret_cast<float*>(own_all);
        const int rows = (p.m - (int)blockIdx.x + p.splits - 1) / p.splits;
        for (int i = threadIdx.x; i < 32 * rows; i += kTcThreads) {
            const int row = blockIdx.x + i / 32 * p.splits, at = 4 * (i % 32), ch = blockIdx.y * 128 + at;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int v = 0; v < p.splits; ++v) {
                const float4 o = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, v) + row * 128 + at);
                sum.x += o.x, sum.y += o.y, sum.z += o.z, sum.w += o.w;
            }
            if (ch >= p.n_out) continue;
            const long long to = (long long)row * p.n_out + ch;
            if (!guard(to + 4 <= (long long)p.m * p.n_out, status)) continue;
            if (p.y_fp32) {
                *reinterpret_cast<float4*>(static_cast<float*>(p.y) + to) = sum;
            } else {
                const __half2 lo = __floats2half2_rn(sum.x, sum.y), hi = __floats2half2_rn(sum.z, sum.w);
                *reinterpret_cast<uint2*>(static_cast<__half*>(p.y) + to) = make_uint2(h2_bits(lo), h2_bits(hi));
            }
        }
        cluster.sync();                                      // no CTA leaves while its part is read
    }
}

// x in the order of the stages' shared memory: per stage and half (64 inputs) N
// rows of 128 bytes, swizzled, K-step by K-step, each of the inputs that a word of
// the packed layout holds.  A thread writes 16 bytes, two pieces of four inputs;
// rows past the last one are zero.
template <int N>
__global__ void __launch_bounds__(256) q4_x_kernel(const uint16_t* x, int m, int k_in, unsigned char* xt, size_t xt_bytes,
                                                   uint32_t* status)
{
    grid_dep_wait();
    grid_dep_launch();                                       // behind the wait: the product may then read its weights at once
    const int i = blockIdx.x * 256 + threadIdx.x, chunk = i & 7, row = (i >> 3) % N, half = i / (8 * N);
    if (half >= k_in / 64) return;
    const int k = 64 * half + 32 * (chunk >> 2) + 4 * ((chunk >> 1) & 1) + 16 * (chunk & 1);
    uint2 lo = make_uint2(0, 0), hi = lo;
    if (row < m && guard((long long)row * k_in + k + 12 <= (long long)m * k_in, status)) {
        const uint2* from = reinterpret_cast<const uint2*>(x + (long long)row * k_in + k);
        lo = from[0];
        hi = from[2];
    }
    const size_t to = (size_t)half * (N * 128) + row * 128 + ((chunk ^ (row & 7)) << 4);
    if (guard(to + 16 <= xt_bytes, status)) *reinterpret_cast<uint4*>(xt + to) = make_uint4(lo.x, lo.y, hi.x, hi.y);
}

template <int N, int GROUP>
cudaError_t launch_t(const Q4TcArgs& a, int blocks, cudaStream_t stream)
{
    using S = Q4Tc<N, GROUP>;
    auto kern = q4_tc_kernel<N, GROUP>;
    static std::atomic<int> done[kMaxDevices];
    const cudaError_t e = once_per_device(done, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    });
    if (e != cudaSuccess) return e;
    const cudaError_t ex = launch_pdl(q4_x_kernel<N>, dim3((unsigned)((a.k_in / 64 * 8 * N + 255) / 256)), dim3(256), 0, stream, a.x,
                                      a.m, a.k_in, const_cast<unsigned char*>(a.xt), a.xt_bytes, reinterpret_cast<uint32_t*>(a.ws));
    if (ex != cudaSuccess) return ex;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)a.splits, (unsigned)blocks);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

struct Q4TcPlan {
    int blocks, splits;
    size_t x_bytes(int m, int k_in) const { return (size_t)(k_in / 64 + 1) / 2 * (m > 16 ? kXStage<32> : kXStage<16>); }
};

// CTAs that share a block of channels are a cluster, of up to four: larger ones
// leave more of the GPU's SMs out.
Q4TcPlan q4_tc_plan(int k_in, int n_out)
{
    const int blocks = (n_out + 127) / 128, stages = (k_in / 64 + 1) / 2;
    const int splits = 148 / blocks < 4 ? 148 / blocks : 4;
    return Q4TcPlan{blocks, splits < 1 ? 1 : splits > stages ? stages : splits};
}

}  // namespace

size_t q4_tc_workspace_bytes(int m, int k_in, int n_out)
{
    return ws_data_off() + q4_tc_plan(k_in, n_out).x_bytes(m, k_in);
}

cudaError_t launch_q4_tc(int m, const uint16_t* x, const uint32_t* packed, const uint16_t* scale, const uint8_t* zero,
                         void* y, int y_fp32, int k_in, int n_out, int group, unsigned char* ws, cudaStream_t stream)
{
    const Q4TcPlan pl = q4_tc_plan(k_in, n_out);
    const Q4TcArgs a = {x, packed, scale, zero, y, m, k_in, n_out, y_fp32 ? 1 : 0, pl.splits, ws, ws + ws_data_off(),
                        pl.x_bytes(m, k_in)};
    if (m <= 16) return group == 64 ? launch_t<16, 64>(a, pl.blocks, stream) : launch_t<16, 128>(a, pl.blocks, stream);
    return group == 32 ? launch_t<32, 32>(a, pl.blocks, stream)
                       : group == 64 ? launch_t<32, 64>(a, pl.blocks, stream) : launch_t<32, 128>(a, pl.blocks, stream);
}

}  // namespace exl3
