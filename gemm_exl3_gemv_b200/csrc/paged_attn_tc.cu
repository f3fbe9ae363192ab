// paged_attn_tc.cu -- the attention of paged_attn.cu for more than 16 rows per
// sequence and head (several drafted tokens x the query heads of a head of the
// cache), on the fifth-generation tensor cores.
//
//     s_t = scale q.k_t,   o = sum_t e^{s_t} v_t / sum_t e^{s_t},   lse = ln sum_t e^{s_t}
//
// Up to 128 rows are the M side of tcgen05.mma (rows past the last one hold
// anything and are not written).  Per 64-token tile:
//   * S = Q K^T (128 x 64, K = head_dim) from shared memory into one of two
//     score buffers in tensor memory, by the MMA warp, one tile ahead;
//   * four softmax warps, a row a thread, read S, mask it, take e^(s - max)
//     with the sum in fp32, and write the probabilities, rounded to fp16, to
//     shared memory in the operand's layout;
//   * O += P V (128 x head_dim, K = 64), the tile's values as the MN-major
//     operand as TMA brought them; its completion frees the tile's stage.
// O stays in tensor memory.  It is rescaled only when a row's maximum has grown
// by more than 2^8 since the last time (the probabilities have that much room
// in fp16, see kUp), which after the first tiles is rare.
// The legacy path of the same rows was bound by shared memory (every 16 rows
// read the tile again) and by the legacy tensor pipe: 66 us for 16 drafted
// tokens of 8 sequences of up to 8192 tokens under a 4096-token window, 40
// query and 8 cache heads.
// Masks: as in paged_attn.cu.  Values that only some rows see and that are not
// finite are added to O by the threads of the rows that see them and cleared
// before the product.
#include "paged_attn.cuh"

namespace exl3 {

namespace {

using namespace attn;

template <int D>
struct ShapeTc {
    static constexpr int kConsumers = 128, kThreads = kConsumers + 64;           // softmax warps; producer and MMA warp
    static constexpr int kRows = 128;
    static constexpr int kHalf = kTile * D * 2;              // bytes of a tile's keys (or values)
    static constexpr int kQ = kRows * D * 2;
    static constexpr int kP = kRows * kTile * 2;             // of one tile
    static constexpr int kRest = kQ + kP + 512;
    static constexpr int kStages = (113 * 1024 - kRest) / (2 * kHalf);           // two CTAs per SM
    static constexpr int kSmem = kStages * 2 * kHalf + kRest;
    static_assert((kThreads + kThreads / 32) * 4 <= kP);     // the fronts lie there until the producer has read them
    static constexpr int kTmemCols = 256;                    // O: D columns from 128 on; S: 64 columns at 0 and at 64
    static constexpr int kSlotRow = D + 4;                   // a row of a partial result: D sums, maximum, sum
    static constexpr int kSlot = kRows * kSlotRow;
    // Probabilities carry a factor 2^kUp (it cancels in o) and are up to 2^kGap
    // over it, 2^15 in all, below fp16's 65504; what is 2^-21 of the maximum is
    // still a normal number, and the rest is off by at most 2^-32 of it.
    static constexpr float kUp = 7.f, kGap = 8.f;
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
        "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// kind::f16, D f32, A and B f16, A K-major, B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn)
{
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void sts16(uint32_t at, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
// 16-byte piece `chunk` of row `row` in 64-column halves of `rows` rows of 128
// bytes, 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int rows, int row, int chunk)
{
    return (chunk >> 3) * (rows * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(ShapeTc<D>::kThreads, 2)
    paged_attn_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnPlan pl,
                         const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using S = ShapeTc<D>;
    extern __shared__ __align__(1024) unsigned char smem[];          // the swizzle counts rows from 1024-byte borders
    unsigned char* q_smem = smem + S::kStages * 2 * S::kHalf;
    unsigned char* p_smem = q_smem + S::kQ;
    int* front = reinterpret_cast<int*>(p_smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(p_smem + S::kP);
    uint64_t* empty = full + S::kStages;
    uint64_t* told = empty + S::kStages;
    uint64_t* heard = told + 2;
    uint64_t* s_full = heard + 2;                            // scores of a buffer are there, are read
    uint64_t* s_free = s_full + 2;
    uint64_t* p_full = s_free + 2;                           // a tile's probabilities are there, their product is done
    uint64_t* pv_done = p_full + 1;
    uint64_t* q_full = pv_done + 1;
    uint64_t* all_done = q_full + 1;
    Stretch* notes = reinterpret_cast<Stretch*>(all_done + 1);
    // whether this CTA is a group's last to arrive; tile whose stretch's O begins with values that are not finite
    int* flags = reinterpret_cast<int*>(notes + 2);
    uint32_t* tmem_base = reinterpret_cast<uint32_t*>(flags + 2);
    static_assert((2 * S::kStages + 12) * 8 + 2 * sizeof(Stretch) + 12 <= 512);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(told + i, 1);
            mbar_init(heard + i, 5);
            mbar_init(s_full + i, 1);
            mbar_init(s_free + i, 4);
        }
        mbar_init(p_full, 4);
        mbar_init(pv_done, 1);
        mbar_init(q_full, 4);
        mbar_init(all_done, 1);
        fence_mbar_init();
        flags[1] = 0;
    }
    grid_dep_wait();
    grid_dep_launch();
    const int total = count_tiles<S::kThreads>(a, pl, front, front + S::kThreads);
    if (total == 0) return;
    const AttnCut cut(total, gridDim.x, pl.least);
    if ((int)blockIdx.x >= cut.ranges) return;
    if (warp == 5) {
        tmem_alloc(tmem_base, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_s = *tmem_base, tmem_o = tmem_s + 128;
    Patience p = {reinterpret_cast<uint32_t*>(a.ws), true};
    const Pipes io = {smem, full, empty, told, heard, notes};

    if (warp == 4) {
        produce<D, S::kStages, S::kThreads>(a, pl, cut, &kmap, &vmap, front, io, p, [](const Stretch&, bool) {});
    } else if (warp == 5) {
        // ------------------------------------------------------ MMA warp ---
        constexpr uint32_t id_qk = idesc_f16(128, kTile, false), id_pv = idesc_f16(128, D, true);
        const uint32_t q_at = smem_u32(q_smem);
        Turn<S::kStages> next, done;                         // tiles whose scores, whose results were asked for
        Turn<2> note, s_buf;
        uint32_t q_phase = 0, p_phase = 0;
        int tile = 0;                                        // of this CTA
        auto result = [&](bool first) {                      // O (+)= P V of the oldest tile without it
            p.wait(p_full, p_phase);
            p_phase ^= 1;
            if (p.alive) {
                tc_fence_after();
                const uint32_t pt = smem_u32(p_smem), vt = smem_u32(smem + done.at * 2 * S::kHalf) + S::kHalf;
                const bool fresh = first && *reinterpret_cast<volatile int*>(flags + 1) != tile;
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_f16_ss_elect(tmem_o, sdesc_sw128(pt + 32 * k, 16, 1024), sdesc_sw128(vt + 2048 * k, kTile * 128, 1024),
                                     id_pv, fresh && k == 0 ? 0u : 1u);
                mma_commit_elect(empty + done.at);
                mma_commit_elect(pv_done);
            }
            done.next();
        };
        while (p.alive) {
            p.wait(told + note.at, note.phase);
            const int n = p.alive ? notes[note.at].n : 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(heard + note.at);
            note.next();
            if (n == 0) break;
            p.wait(q_full, q_phase);
            q_phase ^= 1;
            for (int i = 0; i < n; ++i) {
                p.wait(full + next.at, next.phase);
                p.wait(s_free + s_buf.at, s_buf.phase ^ 1);
                if (p.alive) {
                    tc_fence_after();
                    const uint32_t kt = smem_u32(smem + next.at * 2 * S::kHalf);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_f16_ss_elect(tmem_s + s_buf.at * kTile, sdesc_sw128(q_at + (k >> 2) * (S::kRows * 128) + 32 * (k & 3), 16, 1024),
                                         sdesc_sw128(kt + (k >> 2) * (kTile * 128) + 32 * (k & 3), 16, 1024), id_qk, k > 0 ? 1u : 0u);
                    mma_commit_elect(s_full + s_buf.at);
                }
                next.next();
                s_buf.next();
                ++tile;
                if (i > 0) {
                    --tile;
                    result(i == 1);
                    ++tile;
                }
            }
            result(n == 1);
        }
        mma_commit_elect(all_done);                          // before tensor memory is given back
        (void)mbar_wait_bounded(all_done, 0, 100000000ull);
    } else {
        // ------------------------------------------------- softmax warps ---
        const int row = tid;                                 // and lane of tensor memory
        const uint32_t lanes = (uint32_t)(32 * warp) << 16;
        const auto everyone = [] { named_bar(1, S::kConsumers); };
        Turn<S::kStages> stage;
        Turn<2> note, s_buf;
        int tile = 0, waited = 0;                            // of this CTA
        auto wait_products = [&](int upto) {                 // of the CTA's first `upto` tiles
            for (; waited < upto; ++waited) {
                p.wait(pv_done, waited & 1);
            }
            tc_fence_after();
        };
        while (true) {
            p.wait(told + note.at, note.phase);
            // where a wait of one of the warps has run out all of them leave: none waits for another at a barrier, and
            // how many barriers lie behind this one depends on the note, and on answers that all of them get
            if (named_bar_any(1, S::kConsumers, !p.alive)) break;
            const Stretch st = notes[note.at];
            __syncwarp();
            if (lane == 0) mbar_arrive(heard + note.at);
            note.next();
            if (st.n == 0) break;
            const Entry& en = st.en;

            // this thread's row of queries (the last stretch's products with the queries are done)
            const bool mine = row < en.rows;
            const int rr = en.row0 + (mine ? row : 0), tok = rr / a.group, head = st.h * a.group + rr - tok * a.group;
            const int pos = mine ? en.len - en.count + tok : -1;
            if (mine) {
                const uint4* from = reinterpret_cast<const uint4*>(a.q + st.b * a.q_bs + tok * a.q_rs + (long long)head * D);
                uint4 q[D / 8];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) q[i] = from[i];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) sts16(smem_u32(q_smem) + swizzled(S::kRows, row, i), q[i]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);

            const int p_first = en.len - en.count + en.row0 / a.group;
            const int p_last = en.len - en.count + (en.row0 + en.rows - 1) / a.group;
            const int all_hi = p_first + 1, all_lo = a.window ? p_last - a.window + 1 : 0;
            auto sees = [&](int tk) { return tk <= pos && (!a.window || tk > pos - a.window || tk < a.sinks); };
            auto any_sees = [&](int tk) { return tk <= p_last && (!a.window || tk > p_first - a.window || tk < a.sinks); };
            const int first_tile = tile;
            float mx = kNegInf, sum = 0.f;                   // mx: the maximum when O was last rescaled, in powers of two

            for (int it = 0; it < st.n; ++it, ++tile) {
                const int tok0 = tile_at(en, st.off + it) * kTile;
                p.wait(s_full + s_buf.at, s_buf.phase);
                tc_fence_after();
                uint32_t bits[kTile];
                tmem_ld32(tmem_s + lanes + s_buf.at * kTile, bits);
                tmem_ld32(tmem_s + lanes + s_buf.at * kTile + 32, bits + 32);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free + s_buf.at);
                s_buf.next();
                float s[kTile], scale = pl.scale_log2;       // positive from here on: scores are scaled behind their maximum
#pragma unroll
                for (int j = 0; j < kTile; ++j) s[j] = __uint_as_float(bits[j]);
                if (!(scale > 0.f)) {
#pragma unroll
                    for (int j = 0; j < kTile; ++j) s[j] *= scale;
                    scale = 1.f;
                }
                const uint32_t vt = smem_u32(smem + stage.at * 2 * S::kHalf) + S::kHalf;
                const bool whole = tok0 + kTile <= all_hi && (tok0 >= all_lo || tok0 + kTile <= a.sinks);
                bool odd_values = false;
                if (!whole) {
                    // the tokens this row sees, as bits: [lo, hi) and the sinks
                    const int hi = pos - tok0 + 1, lo = a.window ? pos - a.window - tok0 + 1 : 0, sk = a.sinks - tok0;
#pragma unroll
                    for (int j = 0; j < kTile; ++j) s[j] = j < hi && (j >= lo || j < sk) ? s[j] : kNegInf;
                    // values: what no row of the tile sees is cleared; is there anything that is not finite?
                    p.wait(full + stage.at, stage.phase);
                    bool odd = false;
#pragma unroll 1                                             // two at a time, 128 columns spill: 16 drafted of 8 x 8192 49.7 us, 45.7 so
                    for (int i = tid; i < kTile * (D / 8); i += S::kConsumers) {
                        const int r = i / (D / 8);
                        const uint32_t at = vt + swizzled(kTile, r, i % (D / 8));
                        const uint4 v = lds16(at);
                        if (!any_sees(tok0 + r)) sts16(at, make_uint4(0, 0, 0, 0));
                        else odd |= (finite_halves(v.x) & finite_halves(v.y) & finite_halves(v.z) & finite_halves(v.w)) != 0xffffffffu;
                    }
                    odd_values = named_bar_any(1, S::kConsumers, odd);
                }
                stage.next();

                float tops[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int j = 4; j < kTile; ++j) tops[j & 3] = fmaxf(tops[j & 3], s[j]);
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * scale;
                // the first tile sets the row's maximum; later ones where it has grown too much
                const bool grown = top > mx + S::kGap || mx == kNegInf;
                const float now = grown ? top : mx, cut_at = now == kNegInf ? 0.f : now;
                if (__any_sync(0xffffffffu, grown)) {
                    const float fix = ex2(mx - cut_at);
                    sum *= fix;
                    if (it > 0) {
                        wait_products(tile);                 // of all tiles before this one
#pragma unroll
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(tmem_o + lanes + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fix);
                            tmem_st16(tmem_o + lanes + c, o);
                        }
                        tmem_st_wait();
                    }
                    mx = now;
                }
                const float shift = S::kUp - cut_at;
                float part[4] = {};
#pragma unroll
                for (int j = 0; j < kTile; ++j) {
                    s[j] = ex2(fmaf(s[j], scale, shift));
                    part[j & 3] += s[j];
                }
                sum += (part[0] + part[1]) + (part[2] + part[3]);
                // to the operand's place, once the last product has read it
                wait_products(tile);
                const uint32_t pt = smem_u32(p_smem);
#pragma unroll
                for (int c = 0; c < kTile / 8; ++c)
                    sts16(pt + swizzled(S::kRows, row, c), make_uint4(pack2(s[8 * c], s[8 * c + 1]), pack2(s[8 * c + 2], s[8 * c + 3]),
                                                                     pack2(s[8 * c + 4], s[8 * c + 5]), pack2(s[8 * c + 6], s[8 * c + 7])));
                if (odd_values) {
                    // values that are not finite go to the rows that see them here, and are cleared for the product;
                    // a stretch's first tile then adds to an O that begins with them
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(tmem_o + lanes + c, o);
                        tmem_ld_wait();
                        if (it == 0)
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = 0;
#pragma unroll 1
                        for (int x = 0; x < kTile; ++x) {
                            if (!sees(tok0 + x)) continue;
                            uint32_t pair;
                            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(pair) : "r"(pt + swizzled(S::kRows, row, x >> 3) + 4 * ((x & 7) >> 1)));
                            const float2 pp = __half22float2(*reinterpret_cast<const __half2*>(&pair));
                            const float prob = x & 1 ? pp.y : pp.x;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint4 v4 = lds16(vt + swizzled(kTile, x, c / 8 + i));
                                const uint32_t v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const uint32_t w = v[j] & ~finite_halves(v[j]);
                                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
                                    o[8 * i + 2 * j] = __float_as_uint(__uint_as_float(o[8 * i + 2 * j]) + prob * f.x);
                                    o[8 * i + 2 * j + 1] = __float_as_uint(__uint_as_float(o[8 * i + 2 * j + 1]) + prob * f.y);
                                }
                            }
                        }
                        __syncwarp();
                        tmem_st16(tmem_o + lanes + c, o);
                    }
                    tmem_st_wait();
                    if (it == 0) flags[1] = tile + 1;
                    everyone();
                    for (int i = tid; i < kTile * (D / 8); i += S::kConsumers) {
                        const uint32_t at = vt + swizzled(kTile, i / (D / 8), i % (D / 8));
                        const uint4 v = lds16(at);
                        sts16(at, make_uint4(v.x & finite_halves(v.x), v.y & finite_halves(v.y), v.z & finite_halves(v.z),
                                             v.w & finite_halves(v.w)));
                    }
                }
                fence_proxy_async_smem();                    // probabilities and cleared values, for the tensor cores
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }

            // ---- the stretch's result ----
            wait_products(first_tile + st.n);
            const bool complete = st.n == en.tiles;
            const float inv = pos < 0 ? 0.f : 1.f / sum;     // a row that sees no token: zeros
            float* slot = slot_at<S>(a, st) + row * S::kSlotRow;
            uint16_t* out = a.out + st.b * a.o_bs + tok * a.o_rs + (long long)head * D;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(tmem_o + lanes + c, o);
                tmem_ld_wait();
                if (mine && complete) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t h[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            h[j] = pack2(__uint_as_float(o[i + 2 * j]) * inv, __uint_as_float(o[i + 2 * j + 1]) * inv);
                        *reinterpret_cast<uint4*>(out + c + i) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                } else if (mine) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        __stcg(reinterpret_cast<uint4*>(slot + c + i), make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]));
                }
                __syncwarp();                                // the next read of tensor memory is the whole warp's
            }
            tc_fence_before();                               // read before the next stretch's first product writes there
            if (complete) {
                if (a.lse && mine)
                    a.lse[((long long)st.b * a.m + tok) * a.n_q_heads + head] = pos < 0 ? kNegInf : (mx + (log2f(sum) - S::kUp)) * kLn2;
            } else {
                if (mine) __stcg(reinterpret_cast<float2*>(slot + D), make_float2(mx, sum));
                hand_in<S, D>(a, pl, cut, st, flags[0], tid);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem_s, S::kTmemCols);
    }
}

template <int D>
cudaError_t launch_tc(const AttnArgs& a, const AttnPlan& pl, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream)
{
    using S = ShapeTc<D>;
    auto kern = paged_attn_tc_kernel<D>;
    static std::atomic<int> done[kMaxDevices];
    cudaError_t e = once_per_device(done, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    });
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(kMaxCtas), dim3(S::kThreads), S::kSmem, stream, a, pl, kmap, vmap);
    return e == cudaSuccess && pl.deferred ? launch_join<S, D>(a, pl, stream) : e;
}

}  // namespace

size_t attention_tc_workspace(int head_dim)
{
    return head_dim == 128 ? workspace_of<ShapeTc<128>>() : workspace_of<ShapeTc<64>>();
}

cudaError_t launch_attention_tc(const AttnArgs& a, const AttnPlan& pl, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                cudaStream_t stream)
{
    return a.c.head_dim == 128 ? launch_tc<128>(a, pl, kmap, vmap, stream) : launch_tc<64>(a, pl, kmap, vmap, stream);
}

}  // namespace exl3
