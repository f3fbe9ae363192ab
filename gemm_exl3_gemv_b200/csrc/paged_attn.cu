// paged_attn.cu -- attention of the last few tokens of each sequence over a
// paged key-value cache (exl3_paged_attention).
//
//     s_t = scale q.k_t,   o = sum_t e^{s_t} v_t / sum_t e^{s_t},   lse = ln sum_t e^{s_t}
//
// over the tokens t that a row sees.  With m new tokens and G query heads per
// head of the cache, G m rows share every key and value, so one pass over the
// cache serves them all; at few rows that pass over memory is the bound.
//   * A group is a (sequence, head of the cache, row tile); its work is the
//     64-token tiles its rows see (a window skips the tiles in between).  The
//     tiles of all groups, in order, are cut into equal contiguous ranges, one
//     per CTA, so the lengths may be as ragged as they like.  The cut is worked
//     out on the device from the lengths.
//   * A producer warp brings the tiles to shared memory with TMA (one box per
//     page part and 64 columns, 128-byte swizzle) through a ring; consumer
//     warps run mma.m16n8k16 on them.  The scores stay in registers: running
//     maximum and sum in fp32, probabilities rounded to fp16 as the operand of
//     the second product.
//   * WR warps lie along the rows, WT along the tokens of a tile: with 16 rows
//     or fewer four warps take 16 tokens each and are joined at the end.
//   * A group that several CTAs share is joined by the last of them to arrive,
//     in CTA order.
// Masks.  Tokens past a row's position, outside its window or past the end of
// the sequence must not matter whatever memory holds there.  Scores are
// replaced (not added to); values that no row of the tile sees are cleared in
// the operand; a value that only some rows see and that is not finite goes
// through a separate path that keeps the rows apart.
#include <cuda.h>

#include "exl3_internal.h"
#include "exl3_tc.cuh"

namespace exl3 {

namespace {

constexpr int kTile = 64;                                    // tokens per tile
constexpr float kNegInf = -__builtin_huge_valf();
// Probabilities carry a factor 2^kUp on their way through fp16 (it cancels in
// o): the largest is 2^14, and what is 2^-28 of it is still a normal number.
constexpr float kUp = 14.f;
constexpr float kLn2 = 0.6931471805599453f;
// Tiles per CTA from which another CTA is worth its part of the join.
constexpr int kMinTiles = 4;
constexpr int kFan = 8;                                      // parts joined at once
constexpr int kMaxCtas = 148 * 2;

struct AttnPlan {
    int row_tiles;            // row tiles of a (sequence, head)
    int entries;              // sequences x row tiles
    int page_shift;
    float scale_log2;
};

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
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// 0xffff for each half of the pair that is finite (x * 0 is NaN for the others)
__device__ __forceinline__ uint32_t finite_halves(uint32_t u)
{
    const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&u), __float2half2_rn(0.f));
    return __heq2_mask(z, z);
}
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}

// What an entry (sequence b of the list, row tile) has to do.
struct Entry {
    int seq, len, count;      // len: tokens, the new ones included
    int row0, rows;           // rows of the tile (row r: token r / G, head r % G)
    int sink_tiles;           // leading tiles that only the sinks need
    int tile0;                // first tile of the window
    int tiles;                // all of them
};

__device__ __forceinline__ Entry entry_of(const AttnArgs& a, const AttnPlan& pl, int e, int tile_rows)
{
    Entry r;
    const int b = e / pl.row_tiles, rt = e % pl.row_tiles;
    const int c = a.counts ? min(max(a.counts[b], 0), a.m) : a.m;
    r.seq = a.seqs[b];
    r.count = c;
    r.row0 = rt * tile_rows;
    r.rows = min(c * a.group - r.row0, tile_rows);
    r.sink_tiles = r.tile0 = r.tiles = r.len = 0;
    if (r.seq < 0 || r.seq >= a.c.n_seqs) {
        atomicOr(a.c.scratch + kKvFault, kKvIndex);
        r.rows = 0;
    }
    if (r.rows <= 0) { r.rows = 0; return r; }
    r.len = min(max(a.c.lens[r.seq], 0), a.c.max_pages << pl.page_shift);
    const int p0 = r.len - c + r.row0 / a.group, p1 = r.len - c + (r.row0 + r.rows - 1) / a.group;
    const int hi = max(p1 + 1, 0);                           // tokens [lo, hi) and the sinks
    const int lo = a.window && p0 >= a.window ? p0 - a.window + 1 : 0;
    r.tile0 = lo / kTile;
    r.sink_tiles = min((int)(((long long)a.sinks + kTile - 1) / kTile), r.tile0);
    r.tiles = max(1, r.sink_tiles + (hi + kTile - 1) / kTile - r.tile0);
    return r;
}

__device__ __forceinline__ int tile_at(const Entry& e, int i) { return i < e.sink_tiles ? i : e.tile0 + i - e.sink_tiles; }

__device__ __forceinline__ int cta_of_unit(long long u, long long p, long long total)
{
    return (int)(((u + 1) * p - 1) / total);
}

template <int D, int WR, int WT>
struct AttnShape {
    static constexpr int kConsumers = 32 * WR * WT;
    static constexpr int kThreads = kConsumers + 32;
    static constexpr int kRows = 16 * WR;
    static constexpr int kHalf = kTile * D * 2;              // bytes of a tile's keys (or values)
    static constexpr int kStages = D == 128 ? 3 : 6;
    // shared memory for joining the warps, and the statistics of joined parts
    static constexpr int kJoin = WT > 1 ? (WT / 2) * kRows * (D + 2) * 4 : (kConsumers + kRows) * 8;
    static constexpr int kSmem = kStages * 2 * kHalf + kJoin + 256;   // two CTAs per SM fit
    static constexpr int kSlotRow = D + 4;                   // a row of a partial result: D sums, maximum, sum
    static constexpr int kSlot = kRows * kSlotRow;
};

// Counts the calling CTA in; true in the last of `of` CTAs, which may then read
// what the others wrote before they were counted.  Consumer threads.
__device__ __forceinline__ bool last_of(uint32_t* counter, int of, int& flag, int tid, int threads)
{
    __threadfence();
    named_bar(1, threads);
    if (tid == 0) {
        flag = atomicAdd(counter, 1u) == (uint32_t)of - 1;
        if (flag) *counter = 0;
    }
    named_bar(1, threads);
    const bool last = flag;
    if (last) __threadfence();
    return last;
}

// Parts of a group, joined by the consumers of one CTA in the order of the
// parts: written out (LAST), or to the first part's slot.  First every row's
// maximum and sum, several threads a row; then the weighted sums, a float4 of
// kAcc rows a thread, kDeep parts in flight (the parts lie in the L2; their
// latency is the cost).
template <typename S, int D, bool LAST, typename SlotOf>
__device__ __forceinline__ void join_parts(const AttnArgs& a, const Entry& en, int b, int h, float* slots, int parts,
                                           SlotOf slot_of, float* smem, int tid)
{
    constexpr int kSides = S::kConsumers / S::kRows;
    float2* side = reinterpret_cast<float2*>(smem);
    float2* row_stat = side + S::kConsumers;                 // maximum, 1 / sum
    auto part_of = [&](int c) { return slots + (long long)slot_of(c) * S::kSlot; };
    {
        const int r = tid % S::kRows, first = tid / S::kRows;
        float m = kNegInf, l = 0.f;
#pragma unroll 4
        for (int c = first; c < parts; c += kSides) {
            const float2 ms = __ldcg(reinterpret_cast<const float2*>(part_of(c) + r * S::kSlotRow + D));
            const float now = fmaxf(m, ms.x), c0 = now == kNegInf ? 0.f : now;
            l = l * ex2(m - c0) + ms.y * ex2(ms.x - c0);
            m = now;
        }
        side[tid] = make_float2(m, l);
    }
    named_bar(1, S::kConsumers);
    if (tid < S::kRows) {
        float m = kNegInf, l = 0.f;
#pragma unroll
        for (int i = 0; i < kSides; ++i) {
            const float2 ms = side[i * S::kRows + tid];
            const float now = fmaxf(m, ms.x), c0 = now == kNegInf ? 0.f : now;
            l = l * ex2(m - c0) + ms.y * ex2(ms.x - c0);
            m = now;
        }
        row_stat[tid] = make_float2(m == kNegInf ? 0.f : m, 1.f);
        if constexpr (LAST) {
            const int rr = en.row0 + tid, tok = rr / a.group;
            const bool none = en.len - en.count + tok < 0;   // a row that sees no token: zeros
            row_stat[tid].y = none ? 0.f : 1.f / l;
            if (a.lse && tid < en.rows)
                a.lse[((long long)b * a.m + tok) * a.n_q_heads + h * a.group + rr % a.group] =
                    none ? kNegInf : (m + (log2f(l) - kUp)) * kLn2;
        } else {
            side[tid] = make_float2(m, l);                   // this thread alone reads and writes it from here on
        }
    }
    named_bar(1, S::kConsumers);
    constexpr int kVec = D / 4, kStep = S::kConsumers / kVec;    // rows apart
    constexpr int kAcc = S::kRows / kStep < 4 ? S::kRows / kStep : 4, kDeep = 4;
    const int col = 4 * (tid % kVec);
    for (int r0 = tid / kVec; r0 < S::kRows; r0 += kStep * kAcc) {
        float4 acc[kAcc];
        float top[kAcc];
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            top[i] = row_stat[r0 + i * kStep].x;
        }
        for (int c0 = 0; c0 < parts; c0 += kDeep) {
            float4 v[kDeep][kAcc];
            float w[kDeep][kAcc];
#pragma unroll
            for (int c = 0; c < kDeep; ++c) {
                const float* from = part_of(min(c0 + c, parts - 1));
#pragma unroll
                for (int i = 0; i < kAcc; ++i) {
                    const float* at = from + (r0 + i * kStep) * S::kSlotRow;
                    v[c][i] = __ldcg(reinterpret_cast<const float4*>(at + col));
                    w[c][i] = __ldcg(at + D);
                }
            }
#pragma unroll
            for (int c = 0; c < kDeep; ++c) {
                if (c0 + c >= parts) break;
#pragma unroll
                for (int i = 0; i < kAcc; ++i) {
                    const float f = ex2(w[c][i] - top[i]);
                    acc[i].x += f * v[c][i].x;
                    acc[i].y += f * v[c][i].y;
                    acc[i].z += f * v[c][i].z;
                    acc[i].w += f * v[c][i].w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            const int r = r0 + i * kStep;
            if constexpr (LAST) {
                if (r >= en.rows) break;
                const int rr = en.row0 + r, tok = rr / a.group;
                const float inv = row_stat[r].y;
                *reinterpret_cast<uint2*>(a.out + b * a.o_bs + tok * a.o_rs + (long long)(h * a.group + rr % a.group) * D + col) =
                    make_uint2(pack2(acc[i].x * inv, acc[i].y * inv), pack2(acc[i].z * inv, acc[i].w * inv));
            } else {
                __stcg(reinterpret_cast<float4*>(part_of(0) + r * S::kSlotRow + col), acc[i]);
            }
        }
    }
    named_bar(1, S::kConsumers);
    if constexpr (!LAST)                                     // after every thread has read the first part's maxima
        if (tid < S::kRows) __stcg(reinterpret_cast<float2*>(part_of(0) + tid * S::kSlotRow + D), side[tid]);
}

template <int D, int WR, int WT>
__global__ void __launch_bounds__(AttnShape<D, WR, WT>::kThreads, 2)
    paged_attn_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnPlan pl,
                      const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using S = AttnShape<D, WR, WT>;
    constexpr int TPW = kTile / WT;                          // tokens a warp takes of a tile
    constexpr int NS = TPW / 8;                              // n-tiles of its scores
    constexpr int ND = D / 8;                                // n-tiles of its output
    extern __shared__ __align__(1024) unsigned char smem[];          // the swizzle counts rows from 1024-byte borders
    float* join = reinterpret_cast<float*>(smem + S::kStages * 2 * S::kHalf);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kStages * 2 * S::kHalf + S::kJoin);
    uint64_t* empty = full + S::kStages;
    long long* scan = reinterpret_cast<long long*>(empty + S::kStages);
    long long& first_base = scan[S::kThreads / 32];
    int& first_entry = reinterpret_cast<int*>(&first_base + 1)[0];
    int& last_flag = reinterpret_cast<int*>(&first_base + 1)[1];

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    uint32_t* status = reinterpret_cast<uint32_t*>(a.ws);
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, WR * WT);
        }
        fence_mbar_init();
    }
    grid_dep_wait();
    grid_dep_launch();

    // ---- the cut: this CTA's range [u0, u1) of all tiles ----
    const int heads = a.c.n_heads;
    const int per = (pl.entries + S::kThreads - 1) / S::kThreads;
    const int e_lo = min(pl.entries, tid * per), e_hi = min(pl.entries, e_lo + per);
    long long mine = 0;
    for (int e = e_lo; e < e_hi; ++e) mine += (long long)heads * entry_of(a, pl, e, S::kRows).tiles;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < S::kThreads / 32; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    if (total == 0) return;
    const long long ctas = min((long long)gridDim.x, (total + kMinTiles - 1) / kMinTiles), cta = blockIdx.x;
    if (cta >= ctas) return;
    const long long u0 = total * cta / ctas, u1 = total * (cta + 1) / ctas;
    if (u0 >= before && u0 < before + mine) {
        long long base = before;
        for (int e = e_lo; e < e_hi; ++e) {
            const long long k = (long long)heads * entry_of(a, pl, e, S::kRows).tiles;
            if (u0 < base + k) {
                first_entry = e;
                first_base = base;
                break;
            }
            base += k;
        }
    }
    __syncthreads();

    bool alive = true;                                       // no wait has run out so far
    int stage = 0;
    uint32_t phase = 0;
    int e = first_entry;
    long long base = first_base;

    if (warp == WR * WT) {
        // ---------------------------------------------------- producer ---
        const int ps = 1 << pl.page_shift, parts = ps >= kTile ? 1 : kTile / ps, part_rows = ps < kTile ? ps : kTile;
        for (long long u = u0; u < u1;) {
            const Entry en = entry_of(a, pl, e, S::kRows);
            if (en.tiles == 0) { ++e; continue; }
            const int h = (int)((u - base) / en.tiles), off = (int)((u - base) % en.tiles);
            const int n = (int)min((long long)(en.tiles - off), u1 - u);
            const int* row = a.c.table + (long long)en.seq * a.c.max_pages;
            const int held = (en.len + ps - 1) >> pl.page_shift;
            for (int i0 = 0; i0 < n; i0 += 32 / parts) {
                // each lane looks up the page of one tile part
                const int i = i0 + lane / parts, part = lane % parts;
                int page = -1, token = 0;
                if (i < n) {
                    token = tile_at(en, off + i) * kTile + part * part_rows;
                    const int j = token >> pl.page_shift;
                    if (j < held) {
                        page = row[j];
                        if (page < 0 || page >= a.c.n_pages) {
                            page = -1;
                            atomicOr(a.c.scratch + kKvFault, kKvIndex);
                        }
                    }
                }
                const uint32_t good = __ballot_sync(0xffffffffu, page >= 0);
                for (int k = 0; k < 32 / parts && i0 + k < n; ++k) {
                    if (alive) {
                        alive = mbar_wait_bounded(empty + stage, phase ^ 1);
                        alive = __all_sync(0xffffffffu, alive);
                        if (!alive && lane == 0) atomicOr(status, kStatusTimeout);
                    }
                    if (!alive) continue;                    // no more copies; the consumers give up as well
                    const uint32_t mask = (good >> (k * parts)) & ((1u << parts) - 1);
                    unsigned char* kt = smem + stage * 2 * S::kHalf;
                    if (lane == 0) mbar_arrive_expect_tx(full + stage, __popc(mask) * part_rows * D * 4);
                    __syncwarp();
                    if (lane / parts == k && page >= 0) {
                        const int y = ((page * heads + h) << pl.page_shift) + (token & (ps - 1));
#pragma unroll
                        for (int x = 0; x < D / 64; ++x) {
                            const int at = x * kTile * 128 + part * part_rows * 128;
                            tma_box(kt + at, &kmap, 64 * x, y, full + stage);
                            tma_box(kt + S::kHalf + at, &vmap, 64 * x, y, full + stage);
                        }
                    }
                    __syncwarp();
                    if (++stage == S::kStages) { stage = 0; phase ^= 1; }
                }
            }
            u += n;
            if (u == base + (long long)heads * en.tiles) { base = u; ++e; }
        }
        return;
    }

    // ------------------------------------------------------- consumers ---
    const int wr = warp / WT, wt = warp % WT;
    const int g = lane >> 2, t = lane & 3;
    // lane's row address inside an ldmatrix group: keys 16 tokens x 16 columns, values the same transposed
    const int lm_row = (lane & 7) + ((lane >> 3) & 1) * 8, lm_col = lane >> 4;
    bool first_segment = true;
    for (long long u = u0; u < u1;) {
        const Entry en = entry_of(a, pl, e, S::kRows);
        if (en.tiles == 0) { ++e; continue; }
        const int h = (int)((u - base) / en.tiles), off = (int)((u - base) % en.tiles);
        const int n = (int)min((long long)(en.tiles - off), u1 - u);
        const int b = e / pl.row_tiles;

        // this lane's two rows
        int pos[2];
        const uint16_t* qrow[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = wr * 16 + g + 8 * i;
            const bool ok = r < en.rows;
            const int rr = en.row0 + (ok ? r : 0), tok = rr / a.group;
            pos[i] = ok ? en.len - en.count + tok : -1;
            qrow[i] = ok ? a.q + b * a.q_bs + tok * a.q_rs + (long long)(h * a.group + rr % a.group) * D : nullptr;
        }
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                qf[k][i] = qrow[i & 1] ? *reinterpret_cast<const uint32_t*>(qrow[i & 1] + 16 * k + 2 * t + 8 * (i >> 1)) : 0u;

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

        for (int it = 0; it < n; ++it) {
            const int tok0 = tile_at(en, off + it) * kTile;
            if (alive) {
                alive = mbar_wait_bounded(full + stage, phase);
                alive = __all_sync(0xffffffffu, alive);
                if (!alive && lane == 0) atomicOr(status, kStatusTimeout);
            }
            const uint32_t kt = smem_u32(smem + stage * 2 * S::kHalf), vt = kt + S::kHalf;

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
            if (!whole) {
#pragma unroll
                for (int j = 0; j < NS; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tk = tok0 + wt * TPW + j * 8 + 2 * t + (i & 1), p = pos[i >> 1];
                        s[j][i] = sees(p, tk) ? s[j][i] * pl.scale_log2 : kNegInf;
                    }
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
            float cut[2], fix[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
                const float now = fmaxf(mx[i], top[i]);
                cut[i] = now == kNegInf ? 0.f : now;
                fix[i] = ex2(mx[i] - cut[i]);
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
                    s[j][i] = ex2(s[j][i] - cut[i >> 1] + kUp);
                    sum[i >> 1] += s[j][i];
                }
            // values
            if (whole) {
#pragma unroll
                for (int j = 0; j < NS; j += 2) {
                    const uint32_t pa[4] = {pack2(s[j][0], s[j][1]), pack2(s[j][2], s[j][3]), pack2(s[j + 1][0], s[j + 1][1]),
                                            pack2(s[j + 1][2], s[j + 1][3])};
                    const int row = wt * TPW + j * 8 + lm_row;
#pragma unroll
                    for (int d = 0; d < ND; d += 2) {
                        const int chunk = d + lm_col;
                        uint32_t f[4];
                        ldsm4t(f, vt + (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
                        mma_16816(o[d], pa, f[0], f[1]);
                        mma_16816(o[d + 1], pa, f[2], f[3]);
                    }
                }
            } else {
                uint32_t finite = 0xffffffffu;
#pragma unroll
                for (int j = 0; j < NS; j += 2) {
                    const uint32_t pa[4] = {pack2(s[j][0], s[j][1]), pack2(s[j][2], s[j][3]), pack2(s[j + 1][0], s[j + 1][1]),
                                            pack2(s[j + 1][2], s[j + 1][3])};
                    const int row = wt * TPW + j * 8 + lm_row;
                    // tokens 2t, 2t+1 (0) and 2t+8, 2t+9 (1) of the k-step, which this lane's fragments hold: does any
                    // row of the tile see them?
                    uint32_t keep[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int tk = tok0 + wt * TPW + j * 8 + 2 * t + 8 * i;
                        keep[i] = (any_sees(tk) ? 0xffffu : 0u) | (any_sees(tk + 1) ? 0xffff0000u : 0u);
                    }
#pragma unroll
                    for (int d = 0; d < ND; d += 2) {
                        const int chunk = d + lm_col;
                        uint32_t f[4];
                        ldsm4t(f, vt + (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f[i] &= keep[i & 1];
                            const uint32_t ok = finite_halves(f[i]);
                            finite &= ok;
                            f[i] &= ok;
                        }
                        mma_16816(o[d], pa, f[0], f[1]);
                        mma_16816(o[d + 1], pa, f[2], f[3]);
                    }
                }
                if (__any_sync(0xffffffffu, finite != 0xffffffffu)) {
                    // values that are not finite were left out: only the rows that see them get them
                    for (int x = 0; x < TPW; ++x) {
                        const int tk = tok0 + wt * TPW + x, row = wt * TPW + x;
                        float p[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float mine = 0.f;
#pragma unroll
                            for (int j = 0; j < NS; ++j)
                                if (x >> 3 == j) mine = x & 1 ? s[j][2 * i + 1] : s[j][2 * i];
                            p[i] = __shfl_sync(0xffffffffu, mine, (lane & ~3) | ((x & 7) >> 1));
                        }
                        if (!any_sees(tk)) continue;
#pragma unroll
                        for (int d = 0; d < ND; ++d) {
                            uint32_t v;
                            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v)
                                         : "r"(vt + (d >> 3) * (kTile * 128) + row * 128 + (((d & 7) ^ (row & 7)) << 4) + 4 * t));
                            v &= ~finite_halves(v);
                            const float2 vv = __half22float2(*reinterpret_cast<const __half2*>(&v));
                            if (sees(pos[0], tk)) { o[d][0] += p[0] * vv.x; o[d][1] += p[0] * vv.y; }
                            if (sees(pos[1], tk)) { o[d][2] += p[1] * vv.x; o[d][3] += p[1] * vv.y; }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + stage);
            if (++stage == S::kStages) { stage = 0; phase ^= 1; }
        }

        // the quad's sums
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        }
        // join the warps along the tokens, the upper half into the lower one
#pragma unroll
        for (int half = WT / 2; half >= 1; half /= 2) {
            float* box = join + (wr * (WT / 2) + (wt % half)) * 16 * (D + 2);
            if (wt >= half && wt < 2 * half) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float* at = box + (g + 8 * i) * (D + 2);
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        at[8 * d + 2 * t] = o[d][2 * i];
                        at[8 * d + 2 * t + 1] = o[d][2 * i + 1];
                    }
                    if (t == 0) { at[D] = mx[i]; at[D + 1] = sum[i]; }
                }
            }
            named_bar(1, S::kConsumers);
            if (wt < half) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float* at = box + (g + 8 * i) * (D + 2);
                    const float m2 = at[D], now = fmaxf(mx[i], m2), c0 = now == kNegInf ? 0.f : now;
                    const float f1 = ex2(mx[i] - c0), f2 = ex2(m2 - c0);
                    mx[i] = now;
                    sum[i] = sum[i] * f1 + at[D + 1] * f2;
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        o[d][2 * i] = o[d][2 * i] * f1 + at[8 * d + 2 * t] * f2;
                        o[d][2 * i + 1] = o[d][2 * i + 1] * f1 + at[8 * d + 2 * t + 1] * f2;
                    }
                }
            }
            named_bar(1, S::kConsumers);
        }

        const long long gstart = base + (long long)h * en.tiles;
        if (n == en.tiles) {
            if (wt == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = wr * 16 + g + 8 * i;
                    if (r >= en.rows) continue;
                    const int rr = en.row0 + r, tok = rr / a.group, head = h * a.group + rr % a.group;
                    const float inv = pos[i] < 0 ? 0.f : 1.f / sum[i];    // a row that sees no token: zeros
                    uint16_t* out = a.out + b * a.o_bs + tok * a.o_rs + (long long)head * D;
#pragma unroll
                    for (int d = 0; d < ND; ++d)
                        *reinterpret_cast<uint32_t*>(out + 8 * d + 2 * t) = pack2(o[d][2 * i] * inv, o[d][2 * i + 1] * inv);
                    if (a.lse && t == 0)
                        a.lse[((long long)b * a.m + tok) * a.n_q_heads + head] =
                            pos[i] < 0 ? kNegInf : (mx[i] + (log2f(sum[i]) - kUp)) * kLn2;
                }
            }
        } else {
            // ---- partial result to this CTA's slot; the last CTA of the group joins ----
            float* slots = reinterpret_cast<float*>(a.ws + ws_data_off());
            float* slot = slots + (2 * cta + (first_segment ? 0 : 1)) * S::kSlot;
            if (wt == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float* at = slot + (wr * 16 + g + 8 * i) * S::kSlotRow;
#pragma unroll
                    for (int d = 0; d < ND; ++d)
                        __stcg(reinterpret_cast<float2*>(at + 8 * d + 2 * t), make_float2(o[d][2 * i], o[d][2 * i + 1]));
                    if (t == 0) __stcg(reinterpret_cast<float2*>(at + D), make_float2(mx[i], sum[i]));
                }
            }
            // the group's parts: the first one is its CTA's first or last segment, the others first segments
            const int c_first = cta_of_unit(gstart, ctas, total), c_last = cta_of_unit(gstart + en.tiles - 1, ctas, total);
            const int parts = c_last - c_first + 1, late = gstart == total * c_first / ctas ? 0 : 1;
            auto slot_of = [&](int c) { return 2 * (c_first + c) + (c == 0 ? late : 0); };
            const int mine = (int)cta - c_first;
            // up to kFan parts are joined at once, more in two levels of about the square root
            int fan = parts;
            if (parts > kFan)
                for (fan = kFan / 2; fan * fan < parts; ++fan) {}
            uint32_t* counters = reinterpret_cast<uint32_t*>(a.ws + ws_counter_off());
            const int node = mine / fan * fan, in_node = min(fan, parts - node);
            if (last_of(counters + slot_of(node), in_node, last_flag, tid, S::kConsumers)) {
                if (fan == parts) {
                    join_parts<S, D, true>(a, en, b, h, slots, parts, slot_of, join, tid);
                } else {
                    join_parts<S, D, false>(a, en, b, h, slots, in_node, [&](int c) { return slot_of(node + c); }, join, tid);
                    const int nodes = (parts + fan - 1) / fan;
                    if (last_of(counters + 2 * kMaxCtas + slot_of(0), nodes, last_flag, tid, S::kConsumers))
                        join_parts<S, D, true>(a, en, b, h, slots, nodes, [&](int c) { return slot_of(c * fan); }, join, tid);
                }
            }
        }
        first_segment = false;
        u += n;
        if (u == base + (long long)heads * en.tiles) { base = u; ++e; }
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

// Rows per tile: the smallest that holds a (sequence, head)'s rows, up to 64.
int attn_tile_rows(int m, int group)
{
    const int rows = m * group;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

template <int D, int WR, int WT>
cudaError_t launch_attn_t(const AttnArgs& a, cudaStream_t stream)
{
    using S = AttnShape<D, WR, WT>;
    auto kern = paged_attn_kernel<D, WR, WT>;
    static std::atomic<int> done[kMaxDevices];
    cudaError_t e = once_per_device(done, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    });
    if (e != cudaSuccess) return e;
    EncodeFn fn;
    if ((e = encode_fn(fn)) != cudaSuccess) return e;
    CUtensorMap kmap, vmap;
    if ((e = layer_map(kmap, fn, a.c, a.c.k, a.layer)) != cudaSuccess) return e;
    if ((e = layer_map(vmap, fn, a.c, a.c.v, a.layer)) != cudaSuccess) return e;
    AttnPlan pl;
    pl.row_tiles = (a.m * a.group + S::kRows - 1) / S::kRows;
    pl.entries = a.n * pl.row_tiles;
    pl.page_shift = __builtin_ctz(a.c.page_size);
    pl.scale_log2 = a.scale * 1.4426950408889634f;
    return launch_pdl(kern, dim3(kMaxCtas), dim3(S::kThreads), S::kSmem, stream, a, pl, kmap, vmap);
}

}  // namespace

size_t attention_workspace_bytes(int m, int n_q_heads, int n_heads, int head_dim)
{
    const int rows = attn_tile_rows(m, n_q_heads / n_heads);
    return ws_data_off() + align_up(sizeof(float) * 2 * (size_t)kMaxCtas * rows * (head_dim + 4), 256);
}

cudaError_t launch_paged_attention(const AttnArgs& a, cudaStream_t stream)
{
    const int rows = attn_tile_rows(a.m, a.group);
    if (a.c.head_dim == 128)
        return rows == 16 ? launch_attn_t<128, 1, 4>(a, stream)
                          : rows == 32 ? launch_attn_t<128, 2, 2>(a, stream) : launch_attn_t<128, 4, 1>(a, stream);
    return rows == 16 ? launch_attn_t<64, 1, 4>(a, stream)
                      : rows == 32 ? launch_attn_t<64, 2, 2>(a, stream) : launch_attn_t<64, 4, 1>(a, stream);
}

}  // namespace exl3
