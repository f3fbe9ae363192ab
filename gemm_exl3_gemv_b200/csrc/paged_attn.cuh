// paged_attn.cuh -- what the two attention kernels (paged_attn.cu: up to 16
// rows per sequence and head, paged_attn_tc.cu: more) share: how the work is
// cut, the producer warp that brings it to shared memory, and the join of
// partial results.
//
// A group is a (sequence, head of the cache, row tile); its work is the
// 64-token tiles its rows see (a window skips the tiles in between).  The tiles
// of all groups, in order, are cut into equal contiguous ranges, one per CTA,
// so the lengths may be as ragged as they like; the cut is worked out on the
// device from the lengths.  A group that several CTAs share is joined in the
// order of the ranges: by the last CTA to arrive, or, where that would be a lot
// for one CTA, by a second kernel on the whole GPU (see defer_join()).  (Ranges that CTAs take as they get done were measured too: the
// equal shares of a 131077-token sequence are done between 66 and 100 us, but
// each further stretch cost more than the even finish gave.)
#pragma once
#include <cuda.h>

#include <type_traits>

#include "exl3_cache.h"
#include "exl3_pipe.cuh"
#include "exl3_tc.cuh"

namespace exl3 {

namespace attn {

constexpr int kTile = 64;                                    // tokens per tile
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kFewParts = 8;                                 // of a group, which the last CTA to arrive joins
constexpr int kMaxCtas = 148 * 2;

struct AttnPlan {
    int row_tiles, tile_rows; // row tiles of a (sequence, head), and their rows
    int entries;              // sequences x row tiles
    int page_shift;
    int deferred;             // parts are joined by the second kernel
    int least;                // tiles of a CTA's share
    float scale_log2;
};

// How the tiles of all groups are cut: the first `more` ranges have one tile
// more than `share`.
struct AttnCut {
    int ranges, share, more;
    __device__ __forceinline__ AttnCut(int total, int ctas, int least)
    {
        ranges = min(ctas, (total + least - 1) / least);
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

__device__ __forceinline__ Entry entry_of(const AttnArgs& a, const AttnPlan& pl, int e)
{
    Entry r;
    const int b = e / pl.row_tiles, rt = e % pl.row_tiles;
    int c = a.counts ? a.counts[b] : a.m;
    r.seq = a.seqs[b];
    if (r.seq < 0 || r.seq >= a.c.n_seqs || c < 0 || c > a.m) {
        atomicOr(a.c.scratch + kKvFault, kKvIndex);
        c = 0;
    }
    r.count = c;
    r.row0 = rt * pl.tile_rows;
    r.rows = min(c * a.group - r.row0, pl.tile_rows);
    r.sink_tiles = r.tile0 = r.tiles = r.len = 0;
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

// The tiles in front of every thread's entries, in front[0..THREADS); returns
// all of them.  The whole block; `sums`: a word per warp.
template <int THREADS>
__device__ __forceinline__ int count_tiles(const AttnArgs& a, const AttnPlan& pl, int* front, int* sums)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (pl.entries + THREADS - 1) / THREADS;
    int incl = 0;
    const int e_end = min(pl.entries, (tid + 1) * per);
    for (int e = tid * per; e < e_end; ++e) incl += a.c.n_heads * entry_of(a, pl, e).tiles;
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
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    front[tid] = before;
    __syncthreads();
    return total;
}

// The ring of tiles, and the notes about stretches, in shared memory.
struct Pipes {
    unsigned char* ring;
    uint64_t *full, *empty;              // per stage
    uint64_t *told, *heard;              // two stretches in turn, and when they are read
    Stretch* notes;
};

// The producer warp: walks the CTA's range, tells what the stretches are and
// brings their tiles (TMA, one box per page part and 64 columns, 128-byte
// swizzle).  Its reads of lengths and tables run ahead of the work: with the
// memory saturated, each dependent read takes 2 us.  queries(stretch, allowed):
// called once per stretch, before its tiles.
// A note is written only after the consumers of the one before have said that
// they read it; where that or any other wait runs out, the warp leaves and the
// consumers' own waits run out.  So a note never changes under its readers, and
// all warps of a CTA take the same stretches.  `issued` counts the tiles that it
// sent for.
template <int D, int STAGES, int THREADS, typename Queries>
__device__ __forceinline__ void walk(const AttnArgs& a, const AttnPlan& pl, const AttnCut& cut, const CUtensorMap* kmap,
                                        const CUtensorMap* vmap, const int* front, const Pipes& io, Patience& p, Queries queries,
                                     int& issued)
{
    constexpr int kHalf = kTile * D * 2;                     // bytes of a tile's keys (or values)
    const int lane = threadIdx.x & 31, heads = a.c.n_heads, per = (pl.entries + THREADS - 1) / THREADS;
    Turn<STAGES> stage;
    Turn<2> note;
    // a nonzero injection word, low byte v (tests of the timeout path), lets the first v - 1 tiles through and withholds
    // the others (and the queries of a stretch that begins behind them)
    const uint32_t inject = *reinterpret_cast<const volatile uint32_t*>(a.ws + kWsInjectOff);
    const int most = inject ? max((int)(inject & 255u) - 1, 0) : 0x7fffffff;
    int u = cut.first(blockIdx.x);
    const int u1 = cut.first(blockIdx.x + 1);
    // the entry that tile u belongs to: of the last thread whose entries begin at or in front of it
    int behind = -1;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) behind += __popc(__ballot_sync(0xffffffffu, front[32 * i + lane] <= u));
    int base = front[behind], e = behind * per;
    Entry en = entry_of(a, pl, e);
    const int ps = 1 << pl.page_shift, parts = ps >= kTile ? 1 : kTile / ps, part_rows = ps < kTile ? ps : kTile;
    for (bool first = true; u < u1; first = false) {
        while (u >= base + heads * en.tiles) {
            base += heads * en.tiles;
            en = entry_of(a, pl, ++e);
        }
        const int h = (u - base) / en.tiles, off = (u - base) - h * en.tiles;
        const int n = min(en.tiles - off, u1 - u), b = e / pl.row_tiles;
        p.wait(io.heard + note.at, note.phase ^ 1);
        if (!p.alive) return;
        const Stretch st = {en, b, h, n, off, u - off, first};
        if (lane == 0) {
            io.notes[note.at] = st;
            mbar_arrive(io.told + note.at);
        }
        __syncwarp();
        note.next();
        queries(st, issued < most);
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
                p.wait(io.empty + stage.at, stage.phase ^ 1);
                if (!p.alive) return;
                const bool allowed = issued < most;
                const uint32_t mask = (good >> (k * parts)) & ((1u << parts) - 1);
                unsigned char* kt = io.ring + stage.at * 2 * kHalf;
                if (lane == 0 && allowed) mbar_arrive_expect_tx(io.full + stage.at, __popc(mask) * part_rows * D * 4);
                __syncwarp();
                if (lane / parts == k && page >= 0 && allowed) {
                    const int y = ((page * heads + h) << pl.page_shift) + (token & (ps - 1));
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) {
                        const int at = x * kTile * 128 + part * part_rows * 128;
                        tma_box(kt + at, kmap, 64 * x, y, io.full + stage.at);
                        tma_box(kt + kHalf + at, vmap, 64 * x, y, io.full + stage.at);
                    }
                }
                __syncwarp();
                stage.next();
                issued += allowed;
            }
        }
        u += n;
    }
    p.wait(io.heard + note.at, note.phase ^ 1);
    if (!p.alive) return;
    if (lane == 0) {
        io.notes[note.at].en.rows = 0;
        io.notes[note.at].n = 0;
        mbar_arrive(io.told + note.at);
    }
}

// The producer warp's part of the kernel.
template <int D, int STAGES, int THREADS, typename Queries>
__device__ __forceinline__ void produce(const AttnArgs& a, const AttnPlan& pl, const AttnCut& cut, const CUtensorMap* kmap,
                                        const CUtensorMap* vmap, const int* front, const Pipes& io, Patience& p, Queries queries)
{
    int issued = 0;
    walk<D, STAGES, THREADS>(a, pl, cut, kmap, vmap, front, io, p, queries, issued);
    copies_landed<STAGES>(io.full, issued, p.status);
}

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

// A group cut over several CTAs: its parts are in the slots of consecutive
// ranges' first stretches, but for the first part, which may be its range's
// last stretch (late).
struct Pieces {
    Stretch st;
    int r_first, parts, late;
    __device__ __forceinline__ int slot(int c) const { return 2 * (r_first + c) + (c == 0 ? late : 0); }
};
__device__ __forceinline__ Pieces pieces_of(const AttnCut& cut, const Stretch& st)
{
    Pieces g;
    g.st = st;
    g.r_first = cut.range_of(st.gstart);
    g.parts = cut.range_of(st.gstart + st.en.tiles - 1) - g.r_first + 1;
    g.late = st.gstart == cut.first(g.r_first) ? 0 : 1;
    return g;
}

// In the workspace: two counters (groups on the list, CTAs that are done with
// it) behind the arrival counters, the slots, and the list of cut groups.
__device__ __forceinline__ uint32_t* list_counters(const AttnArgs& a)
{
    return reinterpret_cast<uint32_t*>(a.ws + ws_counter_off()) + kMaxBlocks - 2;
}
__device__ __forceinline__ float* slots_of(const AttnArgs& a) { return reinterpret_cast<float*>(a.ws + ws_data_off()); }
template <typename S>
__device__ __forceinline__ Pieces* list_of(const AttnArgs& a)
{
    return reinterpret_cast<Pieces*>(slots_of(a) + 2ll * kMaxCtas * S::kSlot);
}
template <typename S>
constexpr size_t workspace_of()
{
    return ws_data_off() + align_up(sizeof(float) * 2 * kMaxCtas * S::kSlot + sizeof(Pieces) * kMaxCtas, 256);
}

// Rows base .. of a cut group, joined in the order of the parts and written out
// by THREADS threads.  A thread takes a float4 of ACC rows, with DEEP parts in
// flight (the parts lie in the L2; their latency is the cost), and rescales by
// the rows' maxima as it goes.
template <typename S, int D, int THREADS, int ACC, int DEEP>
__device__ __forceinline__ void join_rows(const AttnArgs& a, const Pieces& g, int base, int tid)
{
    constexpr int kVec = D / 4, kStep = THREADS / kVec;      // rows apart
    const Entry& en = g.st.en;
    const float* slots = slots_of(a);
    const int col = 4 * (tid % kVec), r0 = base + tid / kVec;
    float4 acc[ACC];
    float mx[ACC], sum[ACC];
#pragma unroll
    for (int i = 0; i < ACC; ++i) {
        acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        mx[i] = kNegInf;
        sum[i] = 0.f;
    }
    for (int c0 = 0; c0 < g.parts; c0 += DEEP) {
        float4 v[DEEP][ACC];
        float2 ms[DEEP][ACC];
#pragma unroll
        for (int c = 0; c < DEEP; ++c) {
            const float* from = slots + (long long)g.slot(c0 + c) * S::kSlot;
#pragma unroll
            for (int i = 0; i < ACC; ++i) {
                const float* at = from + (r0 + i * kStep) * S::kSlotRow;
                const bool in = c0 + c < g.parts && r0 + i * kStep < en.rows;
                v[c][i] = in ? __ldcg(reinterpret_cast<const float4*>(at + col)) : make_float4(0.f, 0.f, 0.f, 0.f);
                ms[c][i] = in ? __ldcg(reinterpret_cast<const float2*>(at + D)) : make_float2(kNegInf, 0.f);
            }
        }
#pragma unroll
        for (int i = 0; i < ACC; ++i) {
            float now = mx[i];
#pragma unroll
            for (int c = 0; c < DEEP; ++c) now = fmaxf(now, ms[c][i].x);
            const float at = now == kNegInf ? 0.f : now, f0 = ex2(mx[i] - at);
            mx[i] = now;
            sum[i] *= f0;
            acc[i].x *= f0, acc[i].y *= f0, acc[i].z *= f0, acc[i].w *= f0;
#pragma unroll
            for (int c = 0; c < DEEP; ++c) {
                const float f = ex2(ms[c][i].x - at);
                sum[i] += f * ms[c][i].y;
                acc[i].x += f * v[c][i].x;
                acc[i].y += f * v[c][i].y;
                acc[i].z += f * v[c][i].z;
                acc[i].w += f * v[c][i].w;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ACC; ++i) {
        const int r = r0 + i * kStep;
        if (r >= en.rows) break;
        const int rr = en.row0 + r, tok = rr / a.group, head = g.st.h * a.group + rr - tok * a.group;
        const bool none = en.len - en.count + tok < 0;       // a row that sees no token: zeros
        const float inv = none ? 0.f : 1.f / sum[i];
        *reinterpret_cast<uint2*>(a.out + g.st.b * a.o_bs + tok * a.o_rs + (long long)head * D + col) =
            make_uint2(pack2(acc[i].x * inv, acc[i].y * inv), pack2(acc[i].z * inv, acc[i].w * inv));
        if (a.lse && col == 0)
            a.lse[((long long)g.st.b * a.m + tok) * a.n_q_heads + head] = none ? kNegInf : (mx[i] + (log2f(sum[i]) - S::kUp)) * kLn2;
    }
}

// Where a stretch's partial result goes.
template <typename S>
__device__ __forceinline__ float* slot_at(const AttnArgs& a, const Stretch& st)
{
    return slots_of(a) + (long long)(2 * blockIdx.x + (st.first ? 0 : 1)) * S::kSlot;
}
// After it is there, the consumer threads: the group of the first part goes on
// the list for the second kernel, or the last CTA to arrive joins.
template <typename S, int D>
__device__ __forceinline__ void hand_in(const AttnArgs& a, const AttnPlan& pl, const AttnCut& cut, const Stretch& st, int& flag, int tid)
{
    const Pieces g = pieces_of(cut, st);
    if (pl.deferred) {
        if (tid == 0 && (int)blockIdx.x == g.r_first) list_of<S>(a)[atomicAdd(list_counters(a), 1u)] = g;
        return;
    }
    uint32_t* counter = reinterpret_cast<uint32_t*>(a.ws + ws_counter_off()) + g.slot(0);
    if (!last_of(counter, g.parts, flag, tid, S::kConsumers)) return;
    constexpr int kStep = S::kConsumers / (D / 4), kAcc = S::kRows / kStep < 4 ? S::kRows / kStep : 4;
    static_assert(S::kRows % (kStep * kAcc) == 0);
    for (int base = 0; base < st.en.rows; base += kStep * kAcc) join_rows<S, D, S::kConsumers, kAcc, 4>(a, g, base, tid);
}

// The second kernel: grid (groups that may be cut, rows / kJoinRows).  Few rows
// come in many parts, many rows in a few.
constexpr int kJoinThreads = 128;
template <typename S>
constexpr int kJoinAcc = S::kRows > 16 ? 2 : 1;
template <typename S>
constexpr int kJoinDeep = S::kRows > 16 ? 8 : 16;
template <typename S, int D>
constexpr int kJoinRows = kJoinThreads / (D / 4) * kJoinAcc<S>;
template <typename S, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnArgs a)
{
    __shared__ Pieces g;
    grid_dep_wait();
    grid_dep_launch();
    uint32_t* counters = list_counters(a);
    const bool in = blockIdx.x < *reinterpret_cast<volatile uint32_t*>(counters);
    const int* from = reinterpret_cast<const int*>(list_of<S>(a) + blockIdx.x);    // read before it is known whether there is one
    for (int i = threadIdx.x; i < (int)(sizeof(Pieces) / 4); i += kJoinThreads) reinterpret_cast<int*>(&g)[i] = __ldcg(from + i);
    __syncthreads();
    const int base = blockIdx.y * kJoinRows<S, D>;
    if (in && base < g.st.en.rows) join_rows<S, D, kJoinThreads, kJoinAcc<S>, kJoinDeep<S>>(a, g, base, threadIdx.x);
    if (threadIdx.x == 0 && atomicAdd(counters + 1, 1u) == gridDim.x * gridDim.y - 1) counters[0] = counters[1] = 0;
}

template <typename S, int D>
cudaError_t launch_join(const AttnArgs& a, const AttnPlan& pl, cudaStream_t stream)
{
    const long long groups = (long long)pl.entries * a.c.n_heads;
    const dim3 grid((unsigned)(groups < kMaxCtas ? groups : kMaxCtas), (unsigned)((pl.tile_rows + kJoinRows<S, D> - 1) / kJoinRows<S, D>));
    return launch_pdl(join_kernel<S, D>, grid, dim3(kJoinThreads), 0, stream, a);
}

}  // namespace attn

// The launch of the kernel for more than 16 rows (paged_attn_tc.cu).
cudaError_t launch_attention_tc(const AttnArgs& a, const attn::AttnPlan& pl, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, cudaStream_t stream);
size_t attention_tc_workspace(int head_dim);

}  // namespace exl3
