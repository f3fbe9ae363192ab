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
//   * A producer warp walks the CTA's range.  It brings queries and tiles to
//     shared memory (TMA, one box per page part and 64 columns, 128-byte
//     swizzle, through a ring) and tells the consumers what each stretch of
//     tiles is: with the memory saturated a dependent read costs 2 us, and the
//     producer makes them while earlier tiles are worked on.
//   * WR warps lie along the rows.  With 64 rows or fewer, WT warps share 16
//     rows: each takes some of the tile's tokens for the scores and, after the
//     row maxima and the probabilities went through shared memory, some of the
//     columns of the result, so that nothing has to be joined but sums.
//   * mma.m16n8k16 for both products; running maximum and sum in fp32,
//     probabilities rounded to fp16 as the operand of the second product.
//   * A group that several CTAs share is joined by the last of them to arrive,
//     in the order of the ranges, in two levels when they are many.
// (Ranges that CTAs take as they get done were measured too: the equal shares
// of a 131077-token sequence are done between 66 and 100 us, but each further
// stretch cost more than the even finish gave.)
// Masks.  Tokens past a row's position, outside its window or past the end of
// the sequence must not matter whatever memory holds there.  Scores are
// replaced (not added to); values that no row of the tile sees are cleared in
// shared memory; and values that only some rows see and that are not finite are
// left out of the second product and added to the rows that see them.
#include <cuda.h>

#include <type_traits>

#include "exl3_cache.h"
#include "exl3_tc.cuh"

namespace exl3 {

namespace {

constexpr int kTile = 64;                                    // tokens per tile
constexpr float kNegInf = -__builtin_huge_valf();
// Probabilities carry a factor 2^kUp on their way through fp16 (it cancels in
// o): the largest is 2^14, and what is 2^-28 of it is still a normal number.
constexpr float kUp = 14.f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMinTiles = 2;                                 // of a CTA's share, from which another CTA is worth its part of the join
constexpr int kFan = 8;                                      // parts joined at once
constexpr int kMaxCtas = 148 * 2;

struct AttnPlan {
    int row_tiles;            // row tiles of a (sequence, head)
    int entries;              // sequences x row tiles
    int page_shift;
    float scale_log2;
};

// How the tiles of all groups are cut: the first `more` ranges have one tile
// more than `share`.
struct AttnCut {
    int ranges, share, more;
    __device__ __forceinline__ AttnCut(int total, int ctas)
    {
        ranges = min(ctas, (total + kMinTiles - 1) / kMinTiles);
        share = total / ranges;
        more = total - share * ranges;
    }
    __device__ __forceinline__ int first(int r) const { return r * share + min(r, more); }
    __device__ __forceinline__ int range_of(int tile) const
    {
        const int border = more * (share + 1);
        return tile < border ? tile / (share + 1) : more + (tile - border) / share;
    }
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

// What the producer tells the consumers: the next stretch is n tiles from tile
// off on of head h of an entry, whose group's first tile is gstart.  n = 0:
// there are no more.
struct Stretch {
    Entry en;
    int b, h, n, off, gstart, first;     // first: the first of this CTA's stretches
};

template <int D, int WR, int WT>
struct AttnShape {
    static constexpr int kConsumers = 32 * WR * WT;
    static constexpr int kThreads = kConsumers + 32;
    static constexpr int kRows = 16 * WR;
    static constexpr int kHalf = kTile * D * 2;              // bytes of a tile's keys (or values)
    static constexpr int kPerSm = WR == 1 ? 2 : 1;           // CTAs
    // rows of queries, and of probabilities, lie 16 bytes further apart than
    // they are long: ldmatrix then meets no bank twice
    static constexpr int kQRow = 2 * D + 16, kQ = kRows * kQRow;
    static constexpr int kPRow = 2 * kTile + 16, kP = WT > 1 ? 2 * kRows * kPRow : 0;    // for two tiles in turn
    static constexpr int kTop = WT > 1 ? 2 * kConsumers / 2 : 0;                         // floats: row maxima, in turn
    static constexpr int kFronts = (kThreads + kThreads / 32 + 3) / 4 * 16;              // until the producer has read them
    static constexpr int kRest = kQ + kP + kTop * 4 + kFronts + 512, kRoom = (kPerSm == 2 ? 113 : 227) * 1024 - kRest;
    static constexpr int kStages = kRoom / (2 * kHalf) < 8 ? kRoom / (2 * kHalf) : 8;    // of the ring: as many as fit
    static constexpr int kSmem = kStages * 2 * kHalf + kRest;
    static constexpr int kSlotRow = D + 4;                   // a row of a partial result: D sums, maximum, sum
    static constexpr int kSlot = kRows * kSlotRow;
};

// Counts the calling CTA in; true in the last of `of` CTAs, which may then read
// what the others wrote before they were counted.  Consumer threads: the
// barriers order the other threads' accesses around the first one's fences.
__device__ __forceinline__ bool last_of(uint32_t* counter, int of, int& flag, int tid, int threads)
{
    named_bar(1, threads);
    if (tid == 0) {
        __threadfence();
        flag = atomicAdd(counter, 1u) == (uint32_t)of - 1;
        if (flag) *counter = 0;
        __threadfence();
    }
    named_bar(1, threads);
    return flag;
}

// Parts of a group, joined by the consumers of one CTA in the order of the
// parts: written out (last), or to the first part's slot.  A thread takes a
// float4 of kAcc rows, with kDeep parts in flight (the parts lie in the L2;
// their latency is the cost), and rescales by the rows' maxima as it goes.
template <typename S, int D, typename SlotOf>
__device__ __forceinline__ void join_parts(const AttnArgs& a, const Entry& en, int b, int h, float* slots, int parts,
                                           SlotOf slot_of, bool last, int tid)
{
    constexpr int kVec = D / 4, kStep = S::kConsumers / kVec;    // rows apart
    constexpr int kAcc = S::kRows / kStep < 4 ? S::kRows / kStep : 4, kDeep = 4;
    static_assert(S::kRows % (kStep * kAcc) == 0);
    auto part_of = [&](int c) { return slots + (long long)slot_of(c) * S::kSlot; };
    const int col = 4 * (tid % kVec);
    for (int r0 = tid / kVec; r0 < S::kRows; r0 += kStep * kAcc) {
        float4 acc[kAcc];
        float mx[kAcc], sum[kAcc];
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            mx[i] = kNegInf;
            sum[i] = 0.f;
        }
        for (int c0 = 0; c0 < parts; c0 += kDeep) {
            float4 v[kDeep][kAcc];
            float2 ms[kDeep][kAcc];
#pragma unroll
            for (int c = 0; c < kDeep; ++c) {
                const float* from = part_of(c0 + c);
#pragma unroll
                for (int i = 0; i < kAcc; ++i) {
                    const float* at = from + (r0 + i * kStep) * S::kSlotRow;
                    const bool in = c0 + c < parts;
                    v[c][i] = in ? __ldcg(reinterpret_cast<const float4*>(at + col)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    ms[c][i] = in ? __ldcg(reinterpret_cast<const float2*>(at + D)) : make_float2(kNegInf, 0.f);
                }
            }
#pragma unroll
            for (int i = 0; i < kAcc; ++i) {
                float now = mx[i];
#pragma unroll
                for (int c = 0; c < kDeep; ++c) now = fmaxf(now, ms[c][i].x);
                const float at = now == kNegInf ? 0.f : now, f0 = ex2(mx[i] - at);
                mx[i] = now;
                sum[i] *= f0;
                acc[i].x *= f0, acc[i].y *= f0, acc[i].z *= f0, acc[i].w *= f0;
#pragma unroll
                for (int c = 0; c < kDeep; ++c) {
                    const float f = ex2(ms[c][i].x - at);
                    sum[i] += f * ms[c][i].y;
                    acc[i].x += f * v[c][i].x;
                    acc[i].y += f * v[c][i].y;
                    acc[i].z += f * v[c][i].z;
                    acc[i].w += f * v[c][i].w;
                }
            }
        }
        // row maxima of the first part are read by other threads until here
        if (!last) named_bar(1, S::kConsumers);
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            const int r = r0 + i * kStep;
            if (last) {
                if (r >= en.rows) break;
                const int rr = en.row0 + r, tok = rr / a.group, head = h * a.group + rr - tok * a.group;
                const bool none = en.len - en.count + tok < 0;    // a row that sees no token: zeros
                const float inv = none ? 0.f : 1.f / sum[i];
                *reinterpret_cast<uint2*>(a.out + b * a.o_bs + tok * a.o_rs + (long long)head * D + col) =
                    make_uint2(pack2(acc[i].x * inv, acc[i].y * inv), pack2(acc[i].z * inv, acc[i].w * inv));
                if (a.lse && col == 0)
                    a.lse[((long long)b * a.m + tok) * a.n_q_heads + head] = none ? kNegInf : (mx[i] + (log2f(sum[i]) - kUp)) * kLn2;
            } else {
                float* at = part_of(0) + r * S::kSlotRow;
                __stcg(reinterpret_cast<float4*>(at + col), acc[i]);
                if (col == 0) __stcg(reinterpret_cast<float2*>(at + D), make_float2(mx[i], sum[i]));
            }
        }
    }
}

template <int D, int WR, int WT>
__global__ void __launch_bounds__(AttnShape<D, WR, WT>::kThreads, (AttnShape<D, WR, WT>::kPerSm))
    paged_attn_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnPlan pl,
                      const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using S = AttnShape<D, WR, WT>;
    constexpr int TPW = kTile / WT;                          // tokens whose scores a warp takes
    constexpr int NS = TPW / 8;                              // n-tiles of its scores
    constexpr int CPW = D / WT;                              // columns of the result a warp takes
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
    int* flags = reinterpret_cast<int*>(notes + 2);          // last to arrive; a wait of the consumers has run out
    static_assert((2 * S::kStages + 6) * 8 + 2 * sizeof(Stretch) + 8 <= 512);

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
        for (int i = 0; i < 2; ++i) {
            mbar_init(told + i, 1);
            mbar_init(heard + i, WR * WT);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, WR * WT);
        fence_mbar_init();
        flags[1] = 0;
    }
    grid_dep_wait();
    grid_dep_launch();

    // ---- the tiles in front of every thread's entries, and all of them ----
    const int heads = a.c.n_heads;
    const int per = (pl.entries + S::kThreads - 1) / S::kThreads;
    int* sums = front + S::kThreads;
    int incl = 0;
    const int e_end = min(pl.entries, (tid + 1) * per);
    for (int e = tid * per; e < e_end; ++e) incl += heads * entry_of(a, pl, e, S::kRows).tiles;
    const int mine = incl;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < S::kThreads / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    front[tid] = before;
    __syncthreads();
    if (total == 0) return;
    const AttnCut cut(total, gridDim.x);
    if ((int)blockIdx.x >= cut.ranges) return;

    bool alive = true;                                       // no wait has run out so far
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!alive) return;
        alive = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
        if (!alive && lane == 0) atomicOr(status, kStatusTimeout);
    };
    int stage = 0, note = 0;
    uint32_t phase = 0, note_phase = 0, q_phase = 0;

    if (warp == WR * WT) {
        // ---------------------------------------------------- producer ---
        int u = cut.first(blockIdx.x);
        const int u1 = cut.first(blockIdx.x + 1);
        // the entry that tile u belongs to: of the last thread whose entries begin at or in front of it
        int behind = -1;
#pragma unroll
        for (int i = 0; i < S::kThreads / 32; ++i) behind += __popc(__ballot_sync(0xffffffffu, front[32 * i + lane] <= u));
        int base = front[behind], e = behind * per;
        Entry en = entry_of(a, pl, e, S::kRows);
        const int ps = 1 << pl.page_shift, parts = ps >= kTile ? 1 : kTile / ps, part_rows = ps < kTile ? ps : kTile;
        for (bool first = true; u < u1; first = false) {
            while (u >= base + heads * en.tiles) {
                base += heads * en.tiles;
                en = entry_of(a, pl, ++e, S::kRows);
            }
            const int h = (u - base) / en.tiles, off = (u - base) - h * en.tiles;
            const int n = min(en.tiles - off, u1 - u), b = e / pl.row_tiles;
            wait(heard + note, note_phase ^ 1);
            if (lane == 0) {
                notes[note] = Stretch{en, b, h, n, off, u - off, first};
                mbar_arrive(told + note);
            }
            __syncwarp();
            note ^= 1;
            note_phase ^= note == 0;
            // queries, row by row
            wait(q_empty, q_phase ^ 1);
            q_phase ^= 1;
            if (alive) {
                if (lane == 0) mbar_arrive_expect_tx(q_full, en.rows * 2 * D);
                __syncwarp();
                for (int r = lane; r < en.rows; r += 32) {
                    const int rr = en.row0 + r, tok = rr / a.group;
                    bulk_g2s(q_smem + r * S::kQRow, a.q + b * a.q_bs + tok * a.q_rs + (long long)(h * a.group + rr - tok * a.group) * D,
                             2 * D, q_full);
                }
            }
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
                    wait(empty + stage, phase ^ 1);
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
        }
        wait(heard + note, note_phase ^ 1);
        if (lane == 0) {
            notes[note].n = 0;
            mbar_arrive(told + note);
        }
        return;
    }

    // ------------------------------------------------------- consumers ---
    const int wr = warp / WT, wt = warp % WT;
    const int g = lane >> 2, t = lane & 3;
    // lane's row address inside an ldmatrix group: rows x 16 columns, values the same transposed
    const int lm_row = (lane & 7) + ((lane >> 3) & 1) * 8, lm_col = lane >> 4;
    const auto everyone = [] { named_bar(1, S::kConsumers); };
    const auto row_mates = [&] { named_bar(2 + wr, 32 * WT); };      // the warps that share a row tile
    float* slots = reinterpret_cast<float*>(a.ws + ws_data_off());
    uint32_t* counters = reinterpret_cast<uint32_t*>(a.ws + ws_counter_off());
    while (true) {
        wait(told + note, note_phase);
        if (!alive && lane == 0) flags[1] = 1;
        everyone();
        if (flags[1]) return;                                // all of them: none waits for another at a barrier
        const Stretch st = notes[note];
        __syncwarp();
        if (lane == 0) mbar_arrive(heard + note);
        note ^= 1;
        note_phase ^= note == 0;
        if (st.n == 0) return;
        const Entry& en = st.en;

        uint32_t qf[D / 16][4];
        wait(q_full, q_phase);
        q_phase ^= 1;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) ldsm4(qf[k], smem_u32(q_smem) + (wr * 16 + lm_row) * S::kQRow + 32 * k + 16 * lm_col);
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty);

        // this lane's two rows; rows behind the last hold anything and are not written
        int pos[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = wr * 16 + g + 8 * i;
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
            wait(full + stage, phase);
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
            if constexpr (WT > 1) {
                float* tops = top_smem + (it & 1) * (S::kTop / 2) + wr * (16 * WT);
                if (t == 0) {
                    tops[wt * 16 + g] = top[0];
                    tops[wt * 16 + g + 8] = top[1];
                }
                row_mates();
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int w = 0; w < WT; ++w) top[i] = fmaxf(top[i], tops[w * 16 + g + 8 * i]);
            }
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
                    s[j][i] = ex2(s[j][i] - cut_at[i >> 1] + kUp);
                    sum[i >> 1] += s[j][i];
                }
            // the probabilities as the operand of all 64 tokens
            uint32_t pa[kTile / 16][4];
            const uint32_t p_at = smem_u32(p_smem) + (it & 1) * (S::kP / 2) + wr * (16 * S::kPRow);
            if constexpr (WT > 1) {
#pragma unroll
                for (int j = 0; j < NS; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(p_at + (g + 8 * i) * S::kPRow + 2 * (wt * TPW + j * 8 + 2 * t)),
                                     "r"(pack2(s[j][2 * i], s[j][2 * i + 1])) : "memory");
                row_mates();
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k) ldsm4(pa[k], p_at + lm_row * S::kPRow + 32 * k + 16 * lm_col);
            } else {
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) pa[k][i] = pack2(s[2 * k + (i >> 1)][2 * (i & 1)], s[2 * k + (i >> 1)][2 * (i & 1) + 1]);
            }
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
                    float p[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {            // row g + 8 i of column x of pa
                        uint32_t both = 0;
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            if (x >> 4 == k) both = x & 8 ? pa[k][2 + i] : pa[k][i];
                        both = __shfl_sync(0xffffffffu, both, (lane & ~3) | ((x & 7) >> 1));
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&both));
                        p[i] = x & 1 ? f.y : f.x;
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
                                o[d][2 * i] += p[i] * vv.x;
                                o[d][2 * i + 1] += p[i] * vv.y;
                            }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + stage);
            if (++stage == S::kStages) { stage = 0; phase ^= 1; }
        }

        // the sums of the quad's tokens, and of the row mates'
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        }
        if constexpr (WT > 1) {
            float* tops = top_smem + (st.n & 1) * (S::kTop / 2) + wr * (16 * WT);
            if (t == 0) {
                tops[wt * 16 + g] = sum[0];
                tops[wt * 16 + g + 8] = sum[1];
            }
            row_mates();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sum[i] = 0.f;
#pragma unroll
                for (int w = 0; w < WT; ++w) sum[i] += tops[w * 16 + g + 8 * i];
            }
            row_mates();                                     // read before the next stretch writes there
        }

        if (st.n == en.tiles) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = wr * 16 + g + 8 * i;
                if (r >= en.rows) continue;
                const int rr = en.row0 + r, tok = rr / a.group, head = st.h * a.group + rr - tok * a.group;
                const float inv = pos[i] < 0 ? 0.f : 1.f / sum[i];    // a row that sees no token: zeros
                uint16_t* out = a.out + st.b * a.o_bs + tok * a.o_rs + (long long)head * D + wt * CPW + 2 * t;
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    *reinterpret_cast<uint32_t*>(out + 8 * d) = pack2(o[d][2 * i] * inv, o[d][2 * i + 1] * inv);
                if (a.lse && t == 0 && wt == 0)
                    a.lse[((long long)st.b * a.m + tok) * a.n_q_heads + head] =
                        pos[i] < 0 ? kNegInf : (mx[i] + (log2f(sum[i]) - kUp)) * kLn2;
            }
        } else {
            // ---- partial result to this range's slot; the last CTA of the group joins ----
            float* slot = slots + (long long)(2 * blockIdx.x + (st.first ? 0 : 1)) * S::kSlot;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float* at = slot + (wr * 16 + g + 8 * i) * S::kSlotRow;
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    __stcg(reinterpret_cast<float2*>(at + wt * CPW + 8 * d + 2 * t), make_float2(o[d][2 * i], o[d][2 * i + 1]));
                if (t == 0 && wt == 0) __stcg(reinterpret_cast<float2*>(at + D), make_float2(mx[i], sum[i]));
            }
            // the group's parts: the first one is its range's first or last stretch, the others first ones
            const int r_first = cut.range_of(st.gstart), parts = cut.range_of(st.gstart + en.tiles - 1) - r_first + 1;
            const int late = st.gstart == cut.first(r_first) ? 0 : 1;
            auto slot_of = [&](int c) { return 2 * (r_first + c) + (c == 0 ? late : 0); };
            // up to kFan parts are joined at once, more in two levels of about the square root
            int fan = parts;
            if (parts > kFan)
                for (fan = kFan / 2; fan * fan < parts; ++fan) {}
            const int node = ((int)blockIdx.x - r_first) / fan * fan;
            int from = node, step = 1, count = min(fan, parts - node);
            uint32_t* counter = counters + slot_of(node);
            while (last_of(counter, count, flags[0], tid, S::kConsumers)) {
                const bool last = step == fan || fan == parts;
                join_parts<S, D>(a, en, st.b, st.h, slots, count, [&](int c) { return slot_of(from + c * step); }, last, tid);
                if (last) break;
                from = 0;
                step = fan;
                count = (parts + fan - 1) / fan;
                counter = counters + 2 * kMaxCtas + slot_of(0);
            }
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

// The rows (new tokens x query heads) of a head of the cache are cut into equal
// tiles of up to 128 rows, in 16s; with 64 rows or fewer several warps share 16.
struct AttnRows {
    int row_tiles, warps_r, ctas;
};

AttnRows attn_rows(int m, int group)
{
    AttnRows r;
    const int rows = m * group;
    r.row_tiles = (rows + 127) / 128;
    r.warps_r = ((rows + r.row_tiles - 1) / r.row_tiles + 15) / 16;
    r.ctas = r.warps_r == 1 ? kMaxCtas : kMaxCtas / 2;
    return r;
}
static_assert(4 * kMaxCtas <= kMaxBlocks);                   // two counters a slot

template <int D, int WR, int WT>
cudaError_t launch_attn_t(const AttnArgs& a, const AttnRows& rows, cudaStream_t stream)
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
    pl.row_tiles = rows.row_tiles;
    pl.entries = a.n * pl.row_tiles;
    pl.page_shift = __builtin_ctz(a.c.page_size);
    pl.scale_log2 = a.scale * 1.4426950408889634f;
    return launch_pdl(kern, dim3((unsigned)rows.ctas), dim3(S::kThreads), S::kSmem, stream, a, pl, kmap, vmap);
}

template <int D>
cudaError_t launch_attn_d(const AttnArgs& a, const AttnRows& rows, cudaStream_t stream)
{
    switch (rows.warps_r) {
        case 1: return launch_attn_t<D, 1, 4>(a, rows, stream);
        case 2: return launch_attn_t<D, 2, 4>(a, rows, stream);
        case 3: return launch_attn_t<D, 3, 4>(a, rows, stream);
        case 4: return launch_attn_t<D, 4, 2>(a, rows, stream);
        case 5: return launch_attn_t<D, 5, 2>(a, rows, stream);
        case 6: return launch_attn_t<D, 6, 2>(a, rows, stream);
        case 7: return launch_attn_t<D, 7, 2>(a, rows, stream);
        default: return launch_attn_t<D, 8, 1>(a, rows, stream);
    }
}

}  // namespace

size_t attention_workspace_bytes(int m, int n_q_heads, int n_heads, int head_dim)
{
    const AttnRows r = attn_rows(m, n_q_heads / n_heads);
    return ws_data_off() + align_up(sizeof(float) * 2 * (size_t)r.ctas * 16 * r.warps_r * (head_dim + 4), 256);
}

bool attention_tiles_ok(const AttnArgs& a)
{
    const AttnRows r = attn_rows(a.m, a.group);
    const long long tokens = (long long)a.c.max_pages * a.c.page_size;
    return (long long)a.n * r.row_tiles * a.c.n_heads * (tokens / kTile + 2) < (1ll << 31) - (1 << 20);
}

cudaError_t launch_paged_attention(const AttnArgs& a, cudaStream_t stream)
{
    const AttnRows rows = attn_rows(a.m, a.group);
    return a.c.head_dim == 128 ? launch_attn_d<128>(a, rows, stream) : launch_attn_d<64>(a, rows, stream);
}

}  // namespace exl3
