// paged_attn.cu -- attention of the last few tokens of each sequence over a
// paged key-value cache (exl3_paged_attention).
//
//     s_t = scale q.k_t,   o = sum_t e^{s_t} v_t / sum_t e^{s_t},   lse = ln sum_t e^{s_t}
//
// over the tokens t that a row sees.  With m new tokens and G query heads per
// head of the cache, G m rows share every key and value, so one pass over the
// cache serves them all; at few rows that pass over memory is the bound.
// This kernel takes up to 16 rows (G m <= 16; paged_attn_tc.cu takes more): four
// consumer warps share them.  Each takes 16 of a tile's 64 tokens for the scores
// and, after the row maxima and the probabilities went through shared memory, a
// quarter of the columns of the result, so that nothing has to be joined but
// sums.  mma.m16n8k16 for both products, which at 16 rows keep a sixth of the
// legacy tensor pipe busy; running maximum and sum in fp32, probabilities
// rounded to fp16 as the operand of the second product.  Two CTAs per SM with
// three stages of 32 KB each keep 192 KB on their way, twice what the latency
// asks for at the memory's rate.  (paged_attn.cuh: the cut of the work, the
// producer warp, the join.)
// Masks.  Tokens past a row's position, outside its window or past the end of
// the sequence must not matter whatever memory holds there.  Scores are
// replaced (not added to); values that no row of the tile sees are cleared in
// shared memory; and values that only some rows see and that are not finite are
// left out of the second product and added to the rows that see them.
#include "paged_attn.cuh"

namespace exl3 {

namespace {

using namespace attn;

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
template <int D>
struct Shape16 {
    static constexpr int kWarps = 4, kConsumers = 32 * kWarps, kThreads = kConsumers + 32;
    static constexpr int kRows = 16;
    static constexpr int kHalf = kTile * D * 2;              // bytes of a tile's keys (or values)
    // rows of queries, and of probabilities, lie 16 bytes further apart than
    // they are long: ldmatrix then meets no bank twice
    static constexpr int kQRow = 2 * D + 16, kQ = kRows * kQRow;
    static constexpr int kPRow = 2 * kTile + 16, kP = 2 * kRows * kPRow;         // for two tiles in turn
    static constexpr int kTop = 2 * kWarps * kRows;                              // floats: row maxima, in turn
    static constexpr int kFronts = (kThreads + kThreads / 32 + 3) / 4 * 16;      // until the producer has read them
    static constexpr int kRest = kQ + kP + kTop * 4 + kFronts + 512;
    static constexpr int kStages = (113 * 1024 - kRest) / (2 * kHalf);           // two CTAs per SM
    static constexpr int kSmem = kStages * 2 * kHalf + kRest;
    static constexpr int kSlotRow = D + 4;                   // a row of a partial result: D sums, maximum, sum
    static constexpr int kSlot = kRows * kSlotRow;
    // Probabilities carry a factor 2^kUp on their way through fp16 (it cancels
    // in o): the largest is 2^14, and what is 2^-28 of it is still a normal
    // number.
    static constexpr float kUp = 14.f;
};

template <int D>
__global__ void __launch_bounds__(Shape16<D>::kThreads, 2)
    paged_attn_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnPlan pl,
                      const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using S = Shape16<D>;
    constexpr int TPW = kTile / S::kWarps;                   // tokens whose scores a warp takes
    constexpr int NS = TPW / 8;                              // n-tiles of its scores
    constexpr int CPW = D / S::kWarps;                       // columns of the result a warp takes
    constexpr int ND = CPW / 8;                              // n-tiles of its result
    extern __shared__ __align__(1024) unsigned char smem[];          // the swizzle counts rows from 1024-byte borders
    unsigned char* q_smem = smem + S::kStages * 2 * S::kHalf;
    unsigned char* p_smem = q_smem + S::kQ;
    float* top_smem = reinterpret_cast<float*>(p_smem + S::kP);
    int* front = reinterpret_cast<int*>(top_smem + S::kTop);
    uint64_t* full = reinterpret_cast<uint64_t*>(front + S::kFronts / 4);
    uint64_t* empty = full + S::kStages;
    uint64_t* told = empty + S::kStages;                     // two stretches in turn, and when they are read
    uint64_t* heard = told + 2;
    uint64_t* q_full = heard + 2;
    uint64_t* q_empty = q_full + 1;
    Stretch* notes = reinterpret_cast<Stretch*>(q_empty + 1);
    int& last = *reinterpret_cast<int*>(notes + 2);          // whether this CTA is a group's last to arrive
    static_assert((2 * S::kStages + 6) * 8 + 2 * sizeof(Stretch) + 4 <= 512);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, S::kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(told + i, 1);
            mbar_init(heard + i, S::kWarps);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, S::kWarps);
        fence_mbar_init();
    }
    grid_dep_wait();
    grid_dep_launch();

    const int total = count_tiles<S::kThreads>(a, pl, front, front + S::kThreads);
    if (total == 0) return;
    const AttnCut cut(total, gridDim.x, pl.least);
    if ((int)blockIdx.x >= cut.ranges) return;

    Patience p = {reinterpret_cast<uint32_t*>(a.ws), true};
    const Pipes io = {smem, full, empty, told, heard, notes};
    uint32_t q_phase = 0;
    if (warp == S::kWarps) {
        int asked = 0;                                       // stretches whose queries were sent for
        produce<D, S::kStages, S::kThreads>(a, pl, cut, &kmap, &vmap, front, io, p, [&](const Stretch& st, bool allowed) {
            p.wait(q_empty, q_phase ^ 1);
            q_phase ^= 1;
            if (!p.alive || !allowed) return;
            ++asked;
            if (lane == 0) mbar_arrive_expect_tx(q_full, st.en.rows * 2 * D);
            __syncwarp();
            if (lane < st.en.rows) {                         // row by row
                const int rr = st.en.row0 + lane, tok = rr / a.group;
                bulk_g2s(q_smem + lane * S::kQRow,
                         a.q + st.b * a.q_bs + tok * a.q_rs + (long long)(st.h * a.group + rr - tok * a.group) * D, 2 * D, q_full);
            }
        });
        copies_landed<1>(q_full, asked, p.status);
        return;
    }

    // ------------------------------------------------------- consumers ---
    const int wt = warp, g = lane >> 2, t = lane & 3;
    // lane's row address inside an ldmatrix group: rows x 16 columns, values the same transposed
    const int lm_row = (lane & 7) + ((lane >> 3) & 1) * 8, lm_col = lane >> 4;
    const auto everyone = [] { named_bar(1, S::kConsumers); };
    Turn<S::kStages> stage;
    Turn<2> note;
    while (true) {
        p.wait(told + note.at, note.phase);
        // where a wait of one of the warps has run out all of them leave: none waits for another at a barrier, and how
        // many barriers lie behind this one depends on the note alone
        if (named_bar_any(1, S::kConsumers, !p.alive)) return;
        const Stretch st = notes[note.at];
        __syncwarp();
        if (lane == 0) mbar_arrive(heard + note.at);
        note.next();
        if (st.n == 0) return;
        const Entry& en = st.en;

        uint32_t qf[D / 16][4];
        p.wait(q_full, q_phase);
        q_phase ^= 1;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) ldsm4(qf[k], smem_u32(q_smem) + lm_row * S::kQRow + 32 * k + 16 * lm_col);
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty);

        // this lane's two rows; rows behind the last hold anything and are not written
        int pos[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = g + 8 * i;
            pos[i] = r < en.rows ? en.len - en.count + (en.row0 + r) / a.group : -1;
        }
        float o[ND][4], mx[2] = {kNegInf, kNegInf}, sum[2] = {0.f, 0.f};
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[d][i] = 0.f;

        // tokens every row of the tile sees: [all_lo, all_hi) and the sinks before all_hi
        const int p_first = en.len - en.count + en.row0 / a.group;
        const int p_last = en.len - en.count + (en.row0 + en.rows - 1) / a.group;
        const int all_hi = p_first + 1, all_lo = a.window ? p_last - a.window + 1 : 0;
        auto sees = [&](int p, int tk) { return tk <= p && (!a.window || tk > p - a.window || tk < a.sinks); };
        auto any_sees = [&](int tk) { return tk <= p_last && (!a.window || tk > p_first - a.window || tk < a.sinks); };

        for (int it = 0; it < st.n; ++it) {
            const int tok0 = tile_at(en, st.off + it) * kTile;
            p.wait(full + stage.at, stage.phase);
            const uint32_t kt = smem_u32(smem + stage.at * 2 * S::kHalf), vt = kt + S::kHalf;

            // scores
            float s[NS][4];
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[j][i] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const int chunk = 2 * k + lm_col;            // 16-byte piece of the row
#pragma unroll
                for (int j = 0; j < NS; j += 2) {
                    const int row = wt * TPW + j * 8 + lm_row;
                    uint32_t f[4];
                    ldsm4(f, kt + (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
                    mma_16816(s[j], qf[k], f[0], f[2]);
                    mma_16816(s[j + 1], qf[k], f[1], f[3]);
                }
            }
            const bool whole = tok0 + kTile <= all_hi && (tok0 >= all_lo || tok0 + kTile <= a.sinks);
            bool odd_values = false;
            if (!whole) {
#pragma unroll
                for (int j = 0; j < NS; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[j][i] = sees(pos[i >> 1], tok0 + wt * TPW + j * 8 + 2 * t + (i & 1)) ? s[j][i] * pl.scale_log2 : kNegInf;
                // this warp's columns: what no row of the tile sees is cleared; is there anything that is not finite?
                bool odd = false;
#pragma unroll 1
                for (int i = lane; i < kTile * ND; i += 32) {
                    const int row = i / ND, chunk = wt * ND + i % ND;
                    const uint32_t at = vt + (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
                    uint32_t v[4];
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at));
                    if (!any_sees(tok0 + row)) asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
                    else odd |= (finite_halves(v[0]) & finite_halves(v[1]) & finite_halves(v[2]) & finite_halves(v[3])) != 0xffffffffu;
                }
                fence_proxy_async_smem();                    // before the next copy to this stage
                odd_values = __any_sync(0xffffffffu, odd);
                __syncwarp();                                // the cleared values are there for every lane
            } else {
#pragma unroll
                for (int j = 0; j < NS; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[j][i] *= pl.scale_log2;
            }
            // running maximum and sum
            float top[2] = {kNegInf, kNegInf};
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) top[i >> 1] = fmaxf(top[i >> 1], s[j][i]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
            }
            float* tops = top_smem + (it & 1) * (S::kTop / 2);
            if (t == 0) {
                tops[wt * 16 + g] = top[0];
                tops[wt * 16 + g + 8] = top[1];
            }
            everyone();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int w = 0; w < S::kWarps; ++w) top[i] = fmaxf(top[i], tops[w * 16 + g + 8 * i]);
            float cut_at[2], fix[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float now = fmaxf(mx[i], top[i]);
                cut_at[i] = now == kNegInf ? 0.f : now;
                fix[i] = ex2(mx[i] - cut_at[i]);
                mx[i] = now;
                sum[i] *= fix[i];
            }
            if (__any_sync(0xffffffffu, fix[0] != 1.f || fix[1] != 1.f)) {
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[d][i] *= fix[i >> 1];
            }
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[j][i] = ex2(s[j][i] - cut_at[i >> 1] + S::kUp);
                    sum[i >> 1] += s[j][i];
                }
            // the probabilities as the operand of all 64 tokens
            uint32_t pa[kTile / 16][4];
            const uint32_t p_at = smem_u32(p_smem) + (it & 1) * (S::kP / 2);
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(p_at + (g + 8 * i) * S::kPRow + 2 * (wt * TPW + j * 8 + 2 * t)),
                                 "r"(pack2(s[j][2 * i], s[j][2 * i + 1])) : "memory");
            everyone();
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) ldsm4(pa[k], p_at + lm_row * S::kPRow + 32 * k + 16 * lm_col);
            // values
            auto product = [&](auto all_finite) {
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k) {
                    const int row = 16 * k + lm_row;
#pragma unroll
                    for (int d = 0; d < ND; d += 2) {
                        const int chunk = wt * ND + d + lm_col;
                        uint32_t f[4];
                        ldsm4t(f, vt + (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
                        if constexpr (!decltype(all_finite)::value)
#pragma unroll
                            for (int i = 0; i < 4; ++i) f[i] &= finite_halves(f[i]);
                        mma_16816(o[d], pa[k], f[0], f[1]);
                        mma_16816(o[d + 1], pa[k], f[2], f[3]);
                    }
                }
            };
            if (!odd_values) {
                product(std::true_type{});
            } else {
                product(std::false_type{});
                // the values left out, token by token: only the rows that see them get them
                for (int x = 0; x < kTile; ++x) {
                    const int tk = tok0 + x;
                    float prob[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {            // row g + 8 i of column x of pa
                        uint32_t both = 0;
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            if (x >> 4 == k) both = x & 8 ? pa[k][2 + i] : pa[k][i];
                        both = __shfl_sync(0xffffffffu, both, (lane & ~3) | ((x & 7) >> 1));
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&both));
                        prob[i] = x & 1 ? f.y : f.x;
                    }
                    const bool see[2] = {sees(pos[0], tk), sees(pos[1], tk)};
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        const int chunk = wt * ND + d;
                        uint32_t v;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v)
                                     : "r"(vt + (chunk >> 3) * (kTile * 128) + x * 128 + (((chunk & 7) ^ (x & 7)) << 4) + 4 * t));
                        v &= ~finite_halves(v);
                        const float2 vv = __half22float2(*reinterpret_cast<const __half2*>(&v));
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (see[i]) {
                                o[d][2 * i] += prob[i] * vv.x;
                                o[d][2 * i + 1] += prob[i] * vv.y;
                            }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + stage.at);
            stage.next();
        }

        // the sums of the quad's tokens, and of the other warps'
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        }
        float* tops = top_smem + (st.n & 1) * (S::kTop / 2);
        if (t == 0) {
            tops[wt * 16 + g] = sum[0];
            tops[wt * 16 + g + 8] = sum[1];
        }
        everyone();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sum[i] = 0.f;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) sum[i] += tops[w * 16 + g + 8 * i];
        }

        if (st.n == en.tiles) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = g + 8 * i;
                if (r >= en.rows) continue;
                const int rr = en.row0 + r, tok = rr / a.group, head = st.h * a.group + rr - tok * a.group;
                const float inv = pos[i] < 0 ? 0.f : 1.f / sum[i];    // a row that sees no token: zeros
                uint16_t* out = a.out + st.b * a.o_bs + tok * a.o_rs + (long long)head * D + wt * CPW + 2 * t;
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    *reinterpret_cast<uint32_t*>(out + 8 * d) = pack2(o[d][2 * i] * inv, o[d][2 * i + 1] * inv);
                if (a.lse && t == 0 && wt == 0)
                    a.lse[((long long)st.b * a.m + tok) * a.n_q_heads + head] =
                        pos[i] < 0 ? kNegInf : (mx[i] + (log2f(sum[i]) - S::kUp)) * kLn2;
            }
        } else {
            // ---- partial result to this stretch's slot ----
            float* slot = slot_at<S>(a, st);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float* at = slot + (g + 8 * i) * S::kSlotRow;
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    __stcg(reinterpret_cast<float2*>(at + wt * CPW + 8 * d + 2 * t), make_float2(o[d][2 * i], o[d][2 * i + 1]));
                if (t == 0 && wt == 0) __stcg(reinterpret_cast<float2*>(at + D), make_float2(mx[i], sum[i]));
            }
            hand_in<S, D>(a, pl, cut, st, last, tid);
        }
    }
}

// ------------------------------------------------------------------- host ---

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeFn& fn)
{
    static std::atomic<EncodeFn> found{nullptr};
    fn = found.load(std::memory_order_acquire);
    if (fn) return cudaSuccess;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
    fn = reinterpret_cast<EncodeFn>(p);
    found.store(fn, std::memory_order_release);
    return cudaSuccess;
}

// One layer's keys (or values) as a matrix of head_dim columns: boxes of 64
// columns and up to 64 rows of one page and head.
cudaError_t layer_map(CUtensorMap& map, EncodeFn fn, const KvArgs& c, uint16_t* pool, int layer)
{
    const long long rows = (long long)c.n_pages * c.n_heads * c.page_size;
    const cuuint64_t dims[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)c.head_dim * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)(c.page_size < kTile ? c.page_size : kTile)};
    const cuuint32_t one[2] = {1, 1};
    const CUresult r = fn(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, pool + (long long)layer * rows * c.head_dim, dims, strides,
                          box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Row tiles of a (sequence, head): up to 16 rows go to this file's kernel, more
// to the other, in equal tiles of up to 128 rows.  Both run two CTAs per SM.
struct AttnRows {
    int row_tiles, tile_rows;
};

AttnRows attn_rows(int m, int group)
{
    const int rows = m * group;
    if (rows <= 16) return AttnRows{1, 16};
    const int tiles = (rows + 127) / 128;
    return AttnRows{tiles, (rows + tiles - 1) / tiles};
}
static_assert(2 * kMaxCtas + 2 <= kMaxBlocks);               // a counter a slot, and the list's

constexpr int kLeastTiles = 2;                               // of a CTA's share, without the second kernel

// Whether the second kernel joins.  It costs a launch, and about 4 us behind
// the first; one CTA takes 1 to 3 us for the 2 or 3 parts of an ordinary group
// of 16 rows (32 sequences of up to 4000 tokens: 64 us, with the second kernel
// 68), but much longer for many parts (one sequence of 8192 tokens 26 us, 18
// with it; of 131077 106 and 102) or for 6 parts of 80 rows (16 drafted tokens of
// 8 sequences: 62 us, 46).  Short tables are cut into few parts whatever the rows.
bool defer_join(const KvArgs& c, int n, int tile_rows)
{
    const long long tiles = (long long)c.max_pages * c.page_size / kTile + 1;
    if (tiles / kLeastTiles <= kFewParts) return false;
    return tile_rows > 16 || (long long)n * c.n_heads * kFewParts < kMaxCtas;
}

template <int D>
cudaError_t launch_16(const AttnArgs& a, const AttnPlan& pl, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream)
{
    using S = Shape16<D>;
    auto kern = paged_attn_kernel<D>;
    static std::atomic<int> done[kMaxDevices];
    cudaError_t e = once_per_device(done, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    });
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(kMaxCtas), dim3(S::kThreads), S::kSmem, stream, a, pl, kmap, vmap);
    return e == cudaSuccess && pl.deferred ? launch_join<S, D>(a, pl, stream) : e;
}

}  // namespace

size_t attention_workspace_bytes(int m, int n_q_heads, int n_heads, int head_dim)
{
    if (attn_rows(m, n_q_heads / n_heads).tile_rows > 16) return attention_tc_workspace(head_dim);
    return head_dim == 128 ? workspace_of<Shape16<128>>() : workspace_of<Shape16<64>>();
}

int attention_launches(const KvArgs& c, int n, int m, int group)
{
    return defer_join(c, n, attn_rows(m, group).tile_rows) ? 2 : 1;
}

bool attention_tiles_ok(const AttnArgs& a)
{
    const AttnRows r = attn_rows(a.m, a.group);
    const long long tokens = (long long)a.c.max_pages * a.c.page_size;
    return (long long)a.n * r.row_tiles * a.c.n_heads * (tokens / kTile + 2) < (1ll << 31) - (1 << 20);
}

cudaError_t launch_paged_attention(const AttnArgs& a, cudaStream_t stream)
{
    const AttnRows r = attn_rows(a.m, a.group);
    cudaError_t e;
    EncodeFn fn;
    if ((e = encode_fn(fn)) != cudaSuccess) return e;
    CUtensorMap kmap, vmap;
    if ((e = layer_map(kmap, fn, a.c, a.c.k, a.layer)) != cudaSuccess) return e;
    if ((e = layer_map(vmap, fn, a.c, a.c.v, a.layer)) != cudaSuccess) return e;
    // Another CTA for fewer tiles than these costs more in the join than it
    // saves: one sequence of 8192 tokens takes 20, 18 and 18 us with 2, 4 and 8,
    // 16 drafted tokens behind it 40, 34 and 29 us; without the second kernel, one
    // of 100 tokens takes 7, 10 and 16 us.
    const bool deferred = defer_join(a.c, a.n, r.tile_rows);
    const int least = !deferred ? kLeastTiles : r.tile_rows > 16 ? 8 : 4;
    const AttnPlan pl = {r.row_tiles, r.tile_rows, a.n * r.row_tiles, __builtin_ctz(a.c.page_size), deferred, least,
                         a.scale * 1.4426950408889634f};
    if (r.tile_rows > 16) return launch_attention_tc(a, pl, kmap, vmap, stream);
    return a.c.head_dim == 128 ? launch_16<128>(a, pl, kmap, vmap, stream) : launch_16<64>(a, pl, kmap, vmap, stream);
}

}  // namespace exl3
