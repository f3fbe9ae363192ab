// kv_cache.cu -- the bookkeeping and the data moves of a paged key-value cache
// (exl3_kv_* in include/exl3.h): sequences grow, shrink, are forked and freed;
// pages are allocated, copied and compacted; new keys and values are written.
//
// Everything is decided on the device, so that a decode step can be captured
// in a graph.  Which pages are free is one bit each: 100,000 pages are 12.5 KB,
// which a CTA counts through in one pass, and the lowest free page is the same
// whatever the order of the atomics that freed it.  Calls that have to agree
// on something (is the list good? do the pages suffice?) let every CTA work it
// out for itself from data that no CTA of the call changes before the last one
// that matters has read it (see extend for those that do not); no CTA waits for
// another.
#include "exl3_common.cuh"
#include "exl3_cache.h"

namespace exl3 {

namespace {

__device__ __forceinline__ int pages_of(int tokens, int page_size) { return (tokens + page_size - 1) / page_size; }

// Sum of v over the block's threads, and in `before` the sum over the threads
// in front.  `tmp`: 33 ints of shared memory; ends with a barrier.
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int& before, int* tmp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = s;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += tmp[w];
        total += tmp[w];
    }
    before = base + s - v;
    return total;
}

// Marks sequence s in the bitmap `seen`; false if it is out of range or marked
// already.
__device__ __forceinline__ bool mark(uint32_t* seen, int s, int n_seqs)
{
    if (s < 0 || s >= n_seqs) return false;
    return (atomicOr(seen + (s >> 5), 1u << (s & 31)) >> (s & 31) & 1u) == 0;
}

__device__ __forceinline__ bool page_ok(const KvArgs& a, int p) { return p >= 0 && p < a.n_pages; }

// One holder less of page p; the page is free after its last one.
__device__ __forceinline__ void drop_page(const KvArgs& a, int p)
{
    if (atomicSub(a.refs + p, 1) == 1) atomicOr(a.free + (p >> 5), 1u << (p & 31));
}

__device__ __forceinline__ int load_acquire(const int* p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_relaxed(int* p, int v)
{
    asm volatile("st.relaxed.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

__device__ __forceinline__ void fault(const KvArgs& a, int bits) { atomicOr(a.scratch + kKvFault, bits); }

// ------------------------------------------------------------------ reset ---

__global__ void __launch_bounds__(256) kv_reset_kernel(KvArgs a)
{
    grid_dep_wait();
    const long long step = (long long)gridDim.x * blockDim.x, first = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    for (long long i = first; i < (long long)a.n_seqs * a.max_pages; i += step) a.table[i] = -1;
    for (long long i = first; i < a.n_seqs; i += step) a.lens[i] = 0;
    for (long long i = first; i < a.n_pages; i += step) a.refs[i] = 0;
    for (long long i = first; i < (a.n_pages + 31) / 32; i += step) {
        const int left = a.n_pages - 32 * (int)i;
        a.free[i] = left >= 32 ? 0xffffffffu : (1u << left) - 1;
    }
    for (long long i = first; i < kKvLists; i += step) a.scratch[i] = 0;
}

// ----------------------------------------------------------------- extend ---
// Every CTA works out what the whole list needs: per entry, how many pages and
// whether its last page has to be copied first because others hold it too.
// The lowest free pages are given out in the order of the list.  The copies,
// in runs of one layer's and head's tokens, are shared out over the CTAs; the
// last CTA to be done writes the bookkeeping, which the others have read.
// Without copies the first CTA is the only one that stays.
// CTAs that have no run leave without being counted, so they may read what is
// being written.  They must find no more copies than there are, to leave in any
// case (a list that looks refused is left too; only the first CTA, which always
// stays, reports it).  An entry that needs no copy looks so to them as well:
//   * with the old length, its last page is the old one, and the references of a
//     page that one sequence holds do not grow;
//   * with the new length, its last page is that page or one that was free, of
//     which there are 0 or 1 references; its number is in the table before the
//     length is (a fence between the two, and lengths are read with acquire), so
//     that it does not matter what the table held there.
// Counting every CTA in took 1.2 to 1.9 us longer (64 sequences by a token each,
// without copies, 5.4 against 3.7).

constexpr int kExtThreads = 256;
constexpr int kExtPer = kKvMaxList / kExtThreads;            // list entries of a thread, at most

__global__ void __launch_bounds__(kExtThreads) kv_extend_kernel(KvArgs a, int n, int m, const int* seqs, const int* counts)
{
    extern __shared__ uint32_t seen[];                       // n_seqs bits
    __shared__ int tmp[33];
    __shared__ int ahead[kKvMaxList + 1];                    // pages that the entries in front take
    __shared__ int copies[kKvMaxList];                       // entries whose last page is copied, in the list's order
    __shared__ int found, is_last;
    const int tid = threadIdx.x, ps = a.page_size;
    for (int i = tid; i < (a.n_seqs + 31) / 32; i += kExtThreads) seen[i] = 0;
    grid_dep_wait();
    grid_dep_launch();
    const int old_fault = __ldcg(a.scratch + kKvFault);
    __syncthreads();

    // this thread's entries: a contiguous run of the list
    const int per = (n + kExtThreads - 1) / kExtThreads, e0 = min(n, tid * per), e1 = min(n, e0 + per);
    int seq[kExtPer], count[kExtPer], old[kExtPer], need[kExtPer];
    bool copy[kExtPer];
    int needs = 0, copied = 0, bad = 0;
#pragma unroll
    for (int i = 0; i < kExtPer; ++i) {
        need[i] = 0;
        copy[i] = false;
        if (i >= e1 - e0) continue;
        seq[i] = seqs[e0 + i];
        count[i] = counts ? counts[e0 + i] : m;
        if (!mark(seen, seq[i], a.n_seqs) || count[i] < 0 || count[i] > m) { bad |= kKvIndex; continue; }
        old[i] = load_acquire(a.lens + seq[i]);
        if (old[i] < 0 || old[i] > a.max_pages * ps) { bad |= kKvIndex; continue; }
        if (count[i] > a.max_pages * ps - old[i]) { bad |= kKvFull; continue; }
        need[i] = pages_of(old[i] + count[i], ps) - pages_of(old[i], ps);
        if (count[i] > 0 && old[i] % ps) {
            const int p = __ldcg(a.table + (long long)seq[i] * a.max_pages + old[i] / ps);
            if (!page_ok(a, p)) { bad |= kKvIndex; continue; }
            copy[i] = __ldcg(a.refs + p) > 1;
            need[i] += copy[i];
        }
        needs += need[i];
        copied += copy[i];
    }
    int at, copy_at;
    const int total = block_scan<kExtThreads>(needs, at, tmp);
    const int n_copies = block_scan<kExtThreads>(copied, copy_at, tmp);
#pragma unroll
    for (int i = 0; i < kExtPer; ++i) {
        if (i >= e1 - e0) continue;
        ahead[e0 + i] = at;
        at += need[i];
        if (copy[i]) copies[copy_at++] = e0 + i;
    }
    if (tid == 0) ahead[n] = total;
    bad = __syncthreads_or(bad & kKvIndex) ? kKvIndex : __syncthreads_or(bad & kKvFull) ? kKvFull : 0;

    // the free bits of this thread's words, and how many lie in front
    const int words = (a.n_pages + 31) / 32, wper = (words + kExtThreads - 1) / kExtThreads;
    const int w0 = min(words, tid * wper), w1 = min(words, w0 + wper);
    int free_before = 0, have = 0;
    if (!bad && total > 0) {
        for (int w = w0; w < w1; ++w) have += __popc(__ldcg(a.free + w));
        if (block_scan<kExtThreads>(have, free_before, tmp) < total) bad = kKvFull;
    }
    if (bad || old_fault) {
        if (bad && blockIdx.x == 0 && tid == 0) fault(a, bad);
        return;                                              // the same answer in every CTA
    }

    // copies: item (copy, layer, head, key or value)
    const int runs = 2 * a.n_layers * a.n_heads;
    const long long items = (long long)n_copies * runs;
    const int ctas = (int)max(1ll, min((long long)gridDim.x, items));
    if ((int)blockIdx.x >= ctas) return;
    const long long page_vec = (long long)a.n_heads * ps * a.head_dim / 8, layer_vec = page_vec * a.n_pages;
    int from = 0, to = 0, run = 0, last_copy = -1;
    for (long long it = blockIdx.x; it < items; it += ctas) {
        const int c = (int)(it / runs), r = (int)(it % runs), layer = (r >> 1) / a.n_heads, h = (r >> 1) % a.n_heads;
        if (c != last_copy) {
            // the page it goes to: the entry's first, of rank ahead[entry] among the free ones
            const int e = copies[c], rank = ahead[e];
            __syncthreads();
            if (rank >= free_before && rank < free_before + have) {
                int left = rank - free_before, w = w0;
                uint32_t bits = __ldcg(a.free + w);
                for (int k; left >= (k = __popc(bits)); left -= k) bits = __ldcg(a.free + ++w);
                while (left-- > 0) bits &= bits - 1;
                found = 32 * w + __ffs(bits) - 1;
            }
            __syncthreads();
            const int s = seqs[e], len = a.lens[s];
            to = found;
            from = a.table[(long long)s * a.max_pages + len / ps];
            run = (len % ps) * a.head_dim / 8;               // 16-byte pieces
            last_copy = c;
        }
        uint4* base = reinterpret_cast<uint4*>(r & 1 ? a.v : a.k) + layer * layer_vec + (long long)h * ps * a.head_dim / 8;
        const uint4* src = base + from * page_vec;
        uint4* dst = base + to * page_vec;
        for (int x = tid; x < run; x += 4 * kExtThreads) {
            uint4 buf[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (x + i * kExtThreads < run) buf[i] = src[x + i * kExtThreads];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (x + i * kExtThreads < run) dst[x + i * kExtThreads] = buf[i];
        }
    }

    if (ctas > 1) {
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            is_last = atomicAdd(a.scratch + kKvArrived, 1) == ctas - 1;
            if (is_last) a.scratch[kKvArrived] = 0;
            __threadfence();
        }
        __syncthreads();
        if (!is_last) return;
    }
    // ---- the bookkeeping ----
    __syncthreads();                                         // every thread has read the list of copies
    // The lowest `total` free pages are taken: which entry's page is each?  A warp
    // takes its threads' words one after the other, a page a lane.
    const int lane = tid & 31;
    int rank = free_before;
    for (int i = 0; i < wper; ++i) {
        const int w = w0 + i;
        const uint32_t mine = w < w1 && rank < total ? __ldcg(a.free + w) : 0;
        uint32_t todo = __ballot_sync(0xffffffffu, mine != 0);
        for (; todo; todo &= todo - 1) {
            const int from = __ffs(todo) - 1, word = __shfl_sync(0xffffffffu, w, from);
            const uint32_t bits = __shfl_sync(0xffffffffu, mine, from);
            const int r = __shfl_sync(0xffffffffu, rank, from) + __popc(bits & ((1u << lane) - 1));
            const bool taken = (bits >> lane & 1) && r < total;
            if (taken) {
                int e = 0, hi = n;                           // the last entry that begins at or in front of this rank
                while (hi - e > 1) {
                    const int mid = (e + hi) / 2;
                    (ahead[mid] <= r ? e : hi) = mid;
                }
                const int page = 32 * word + lane;
                a.refs[page] = 1;
                const int s = seqs[e], c = counts ? counts[e] : m, len = a.lens[s];
                const int fresh = pages_of(len + c, ps) - pages_of(len, ps), nth = r - ahead[e];
                const bool copied_too = ahead[e + 1] - ahead[e] > fresh;
                if (copied_too && nth == 0) copies[e] = page;    // (the list of copies is done with)
                else a.table[(long long)s * a.max_pages + pages_of(len, ps) + nth - copied_too] = page;
            }
            const uint32_t all = __ballot_sync(0xffffffffu, taken);
            if (lane == 0 && all) atomicAnd(a.free + word, ~all);
        }
        rank += __popc(mine);
    }
    __syncthreads();                                         // the free bits and the old lengths were read
    __threadfence();                                         // the new pages are in the tables before the new lengths are there
#pragma unroll
    for (int i = 0; i < kExtPer; ++i) {
        if (i >= e1 - e0) continue;
        if (copy[i]) {
            int* slot = a.table + (long long)seq[i] * a.max_pages + old[i] / ps;
            drop_page(a, *slot);
            *slot = copies[e0 + i];
        }
        store_relaxed(a.lens + seq[i], old[i] + count[i]);
    }
}

// ------------------------------------------------------------------ write ---
// grid.y: the list's entries.  A thread moves 16 bytes of a key and of a value
// at a time; what the places cost (sequence, length, page: three dependent
// loads) is shared by the pieces of a row through the L1.  Every CTA checks the
// whole list first, as a repeated sequence would be written by two entries in
// no order.  Bound by memory: 2001 tokens of two sequences, 8 heads of 128, take
// 7.2 us (4.6 TB/s), 2665 in all 5.8 (3.7); of one token of 64 sequences, 2.4 us,
// the launch and the chain of reads.

__global__ void __launch_bounds__(256) kv_write_kernel(KvArgs a, int layer, int n, int m, const int* seqs, const int* counts,
                                                       const uint16_t* k_new, const uint16_t* v_new, long long bs,
                                                       long long rs)
{
    extern __shared__ uint32_t seen[];
    for (int i = threadIdx.x; i < (a.n_seqs + 31) / 32; i += blockDim.x) seen[i] = 0;
    grid_dep_wait();
    grid_dep_launch();
    const int b = blockIdx.y, s = seqs[b], c = counts ? counts[b] : m;
    const int old_fault = __ldcg(a.scratch + kKvFault);
    __syncthreads();
    bool bad = false;
    for (int e = threadIdx.x; e < n; e += blockDim.x) bad |= !mark(seen, seqs[e], a.n_seqs) || (counts && (counts[e] < 0 || counts[e] > m));
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && b == 0 && threadIdx.x == 0) fault(a, kKvIndex);
        return;
    }
    if (old_fault) return;
    const int row_vec = a.n_heads * a.head_dim / 8, head_vec = a.head_dim / 8, shift = __ffs(a.page_size) - 1;
    const long long page_el = (long long)a.n_heads * a.page_size * a.head_dim;
    const int* pages = a.table + (long long)s * a.max_pages;
    const int first = a.lens[s] - c;
    // this thread's places in the entry's rows
    const uint32_t at = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
    int row = (int)(at / row_vec), vec = (int)(at % row_vec);
    const int row_step = (int)(step / row_vec), vec_step = (int)(step % row_vec);
    for (; row < c; row += row_step, vec += vec_step) {
        if (vec >= row_vec) {
            vec -= row_vec;
            if (++row >= c) break;
        }
        const int pos = first + row;
        if (pos < 0 || pos >= a.max_pages << shift) { fault(a, kKvIndex); continue; }
        const int page = pages[pos >> shift];
        if (!page_ok(a, page)) { fault(a, kKvIndex); continue; }
        const int head = vec / head_vec;
        const long long to = ((long long)layer * a.n_pages + page) * page_el +
                             ((((long long)head << shift) + (pos & (a.page_size - 1))) * a.head_dim + 8 * (vec - head * head_vec));
        const long long from = b * bs + row * rs + 8 * vec;
        *reinterpret_cast<uint4*>(a.k + to) = *reinterpret_cast<const uint4*>(k_new + from);
        *reinterpret_cast<uint4*>(a.v + to) = *reinterpret_cast<const uint4*>(v_new + from);
    }
}

// --------------------------------------------------------- truncate, fork ---
// One CTA per list entry; each checks the whole list (the lists are what no
// CTA changes), then works on its own sequence's row alone.

__global__ void __launch_bounds__(128) kv_truncate_kernel(KvArgs a, int n, const int* seqs, const int* new_lens)
{
    extern __shared__ uint32_t seen[];
    const int words = (a.n_seqs + 31) / 32, ps = a.page_size;
    for (int i = threadIdx.x; i < words; i += blockDim.x) seen[i] = 0;
    grid_dep_wait();
    grid_dep_launch();
    __syncthreads();
    bool bad = false;
    for (int e = threadIdx.x; e < n; e += blockDim.x) bad |= !mark(seen, seqs[e], a.n_seqs) || (new_lens && new_lens[e] < 0);
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) fault(a, kKvIndex);
        return;
    }
    const int s = seqs[blockIdx.x];
    const int old = min(max(a.lens[s], 0), a.max_pages * ps), now = min(old, new_lens ? new_lens[blockIdx.x] : 0);
    int* row = a.table + (long long)s * a.max_pages;
    for (int j = pages_of(now, ps) + threadIdx.x; j < pages_of(old, ps); j += blockDim.x) {
        if (page_ok(a, row[j])) drop_page(a, row[j]);
        else fault(a, kKvIndex);
        row[j] = -1;
    }
    __syncthreads();                                         // the length was read by every thread
    if (threadIdx.x == 0) a.lens[s] = now;
}

__global__ void __launch_bounds__(128) kv_fork_kernel(KvArgs a, int n, const int* src, const int* dst)
{
    extern __shared__ uint32_t seen[];
    const int words = (a.n_seqs + 31) / 32, ps = a.page_size;
    for (int i = threadIdx.x; i < words; i += blockDim.x) seen[i] = 0;
    grid_dep_wait();
    grid_dep_launch();
    __syncthreads();
    bool bad = false;
    for (int e = threadIdx.x; e < n; e += blockDim.x) bad |= !mark(seen, dst[e], a.n_seqs);
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += blockDim.x) {
        const int s = src[e];
        bad |= s < 0 || s >= a.n_seqs || (seen[s >> 5] >> (s & 31) & 1u);
    }
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) fault(a, kKvIndex);
        return;
    }
    const int s = src[blockIdx.x], d = dst[blockIdx.x];
    const int len = min(max(a.lens[s], 0), a.max_pages * ps);
    const bool taken = a.lens[d] != 0;
    __syncthreads();                                         // before the new length is written
    if (taken) {
        if (threadIdx.x == 0) fault(a, kKvIndex);
        return;
    }
    const int* from = a.table + (long long)s * a.max_pages;
    int* to = a.table + (long long)d * a.max_pages;
    for (int j = threadIdx.x; j < pages_of(len, ps); j += blockDim.x) {
        const int p = from[j];
        if (page_ok(a, p)) atomicAdd(a.refs + p, 1);
        else fault(a, kKvIndex);
        to[j] = p;
    }
    if (threadIdx.x == 0) a.lens[d] = len;
}

// ---------------------------------------------------------------- compact ---
// The used pages behind the border and the free ones before it are ranked and
// paired; then the whole GPU moves the pages and renames them in the tables.
// No page is both a source and a destination, so the moves need no order.
// Pools of up to 32 * kMoveThreads pages (one word of free bits a thread) are
// done in one launch: every CTA ranks for itself, and the last one to have done
// so writes the free bits.  Larger ones rank in a launch of one CTA first
// (8 sequences of 150 tokens: 12.4 us in two launches for the free, fork and
// compact of a pass).

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 8;                               // 16-byte pieces in flight per thread
constexpr int kSmallPool = 32 * kMoveThreads;

__device__ __forceinline__ uint32_t bits_below(int n)        // of a word: those of its first n pages
{
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
}

// Ranks the pages in src and dst (ascending); returns the moves, and the border.
template <int THREADS>
__device__ __forceinline__ int pair_pages(const KvArgs& a, int* src, int* dst, int* tmp, int& border)
{
    const int words = (a.n_pages + 31) / 32, per = (words + THREADS - 1) / THREADS;
    const int w0 = min(words, (int)threadIdx.x * per), w1 = min(words, w0 + per);
    int used = 0, before;
    for (int w = w0; w < w1; ++w) used += __popc(~__ldcg(a.free + w) & bits_below(a.n_pages - 32 * w));
    border = block_scan<THREADS>(used, before, tmp);
    int holes = 0, strays = 0, hole_at, stray_at;            // free pages before the border, used pages behind it
    for (int w = w0; w < w1; ++w) {
        const uint32_t f = __ldcg(a.free + w), lo = bits_below(border - 32 * w);
        holes += __popc(f & lo);
        strays += __popc(~f & bits_below(a.n_pages - 32 * w) & ~lo);
    }
    const int moves = block_scan<THREADS>(holes, hole_at, tmp);
    block_scan<THREADS>(strays, stray_at, tmp);
    for (int w = w0; w < w1; ++w) {
        const uint32_t f = __ldcg(a.free + w), lo = bits_below(border - 32 * w);
        for (uint32_t x = f & lo; x; x &= x - 1) dst[hole_at++] = 32 * w + __ffs(x) - 1;
        for (uint32_t x = ~f & bits_below(a.n_pages - 32 * w) & ~lo; x; x &= x - 1) src[stray_at++] = 32 * w + __ffs(x) - 1;
    }
    __syncthreads();
    return moves;
}

// The moves, the counts and the tables, shared out over the grid.
__device__ __forceinline__ void move_pages(const KvArgs& a, const int* src, const int* dst, int moves, int border)
{
    const int ps = a.page_size, page_vec = a.n_heads * ps * a.head_dim / 8;
    constexpr int kChunk = kMoveThreads * kMovePieces;
    const int chunks = (page_vec + kChunk - 1) / kChunk;
    const long long items = (long long)moves * 2 * a.n_layers * chunks;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        // moves x 2 layers stay below 2^19 2^11
        const uint32_t r = (uint32_t)(it / chunks);
        const int chunk = (int)(it - (long long)r * chunks), half = (int)(r & 1);
        const int layer = (int)((r >> 1) % a.n_layers), mv = (int)((r >> 1) / a.n_layers);
        uint4* base = reinterpret_cast<uint4*>(half ? a.v : a.k) + (long long)layer * a.n_pages * page_vec;
        const uint4* from = base + (long long)src[mv] * page_vec;
        uint4* to = base + (long long)dst[mv] * page_vec;
        uint4 buf[kMovePieces];
        const int x0 = chunk * kChunk + threadIdx.x;
#pragma unroll
        for (int i = 0; i < kMovePieces; ++i)
            if (x0 + i * kMoveThreads < page_vec) buf[i] = from[x0 + i * kMoveThreads];
#pragma unroll
        for (int i = 0; i < kMovePieces; ++i)
            if (x0 + i * kMoveThreads < page_vec) to[x0 + i * kMoveThreads] = buf[i];
    }
    const long long first = (long long)blockIdx.x * kMoveThreads + threadIdx.x, step = (long long)gridDim.x * kMoveThreads;
    for (long long i = first; i < moves; i += step) {
        a.refs[dst[i]] = a.refs[src[i]];
        a.refs[src[i]] = 0;
    }
    const int warps = gridDim.x * (kMoveThreads / 32), lane = threadIdx.x & 31;
    for (int s = (int)(first >> 5); s < a.n_seqs; s += warps) {
        int* row = a.table + (long long)s * a.max_pages;
        const int held = pages_of(min(max(a.lens[s], 0), a.max_pages * ps), ps);
        for (int j = lane; j < held; j += 32) {
            const int p = row[j];
            if (!page_ok(a, p)) fault(a, kKvIndex);
            else if (p >= border) {
                int lo = 0, hi = moves;                      // its place among the sources
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    (src[mid] <= p ? lo : hi) = mid;
                }
                if (lo < moves && src[lo] == p) row[j] = dst[lo];
                else fault(a, kKvIndex);                     // the table names a page that is free
            }
        }
    }
}

__global__ void __launch_bounds__(kPlanThreads) kv_compact_plan_kernel(KvArgs a)
{
    __shared__ int tmp[33];
    grid_dep_wait();
    int* src = a.scratch + kKvLists;
    int border;
    const int moves = pair_pages<kPlanThreads>(a, src, src + (a.n_pages + 1) / 2, tmp, border);
    if (threadIdx.x == 0) {
        a.scratch[kKvMoves] = moves;
        a.scratch[kKvUsed] = border;
    }
}

__device__ __forceinline__ void free_behind(const KvArgs& a, int border, int first, int step)
{
    for (int i = first; i < (a.n_pages + 31) / 32; i += step)
        a.free[i] = bits_below(a.n_pages - 32 * i) & ~bits_below(border - 32 * i);
}

__global__ void __launch_bounds__(kMoveThreads, 4) kv_compact_move_kernel(KvArgs a)
{
    grid_dep_wait();
    const int moves = a.scratch[kKvMoves], border = a.scratch[kKvUsed];
    if (moves == 0) return;
    const int* src = a.scratch + kKvLists;
    free_behind(a, border, blockIdx.x * kMoveThreads + threadIdx.x, gridDim.x * kMoveThreads);
    move_pages(a, src, src + (a.n_pages + 1) / 2, moves, border);
}

__global__ void __launch_bounds__(kMoveThreads, 4) kv_compact_small_kernel(KvArgs a)
{
    __shared__ int tmp[33], src[kSmallPool / 2], dst[kSmallPool / 2], is_last;
    grid_dep_wait();
    grid_dep_launch();
    int border;
    const int moves = pair_pages<kMoveThreads>(a, src, dst, tmp, border);
    if (moves == 0) return;                                  // the same in every CTA
    // counted in as one that has read the free bits; whether it was the last one is asked for behind the moves
    int before = 0;
    if (threadIdx.x == 0) {
        __threadfence();
        before = atomicAdd(a.scratch + kKvArrived, 1);
    }
    move_pages(a, src, dst, moves, border);
    if (threadIdx.x == 0) {
        is_last = before == (int)gridDim.x - 1;
        if (is_last) a.scratch[kKvArrived] = 0;
        __threadfence();
    }
    __syncthreads();
    if (is_last) free_behind(a, border, threadIdx.x, kMoveThreads);
}

size_t seen_bytes(const KvArgs& a) { return sizeof(uint32_t) * (size_t)((a.n_seqs + 31) / 32); }

}  // namespace

cudaError_t launch_kv_reset(const KvArgs& a, cudaStream_t stream)
{
    return launch_pdl(kv_reset_kernel, dim3(148), dim3(256), 0, stream, a);
}

cudaError_t launch_kv_extend(const KvArgs& a, int n, int m, const int* seqs, const int* counts, cudaStream_t stream)
{
    return launch_pdl(kv_extend_kernel, dim3(148 * 3), dim3(kExtThreads), seen_bytes(a), stream, a, n, m, seqs, counts);
}

cudaError_t launch_kv_write(const KvArgs& a, int layer, int n, int m, const int* seqs, const int* counts,
                            const uint16_t* k_new, const uint16_t* v_new, long long batch_stride,
                            long long row_stride, cudaStream_t stream)
{
    const long long blocks = ((long long)m * a.n_heads * a.head_dim / 8 + 255) / 256, most = 148 * 8 / n + 1;
    return launch_pdl(kv_write_kernel, dim3((unsigned)(blocks < most ? blocks : most), (unsigned)n), dim3(256), seen_bytes(a),
                      stream, a, layer, n, m, seqs, counts, k_new, v_new, batch_stride, row_stride);
}

cudaError_t launch_kv_truncate(const KvArgs& a, int n, const int* seqs, const int* new_lens, cudaStream_t stream)
{
    return launch_pdl(kv_truncate_kernel, dim3((unsigned)n), dim3(128), seen_bytes(a), stream, a, n, seqs, new_lens);
}

cudaError_t launch_kv_fork(const KvArgs& a, int n, const int* src, const int* dst, cudaStream_t stream)
{
    return launch_pdl(kv_fork_kernel, dim3((unsigned)n), dim3(128), seen_bytes(a), stream, a, n, src, dst);
}

cudaError_t launch_kv_compact(const KvArgs& a, cudaStream_t stream)
{
    if (a.n_pages <= kSmallPool) return launch_pdl(kv_compact_small_kernel, dim3(148 * 4), dim3(kMoveThreads), 0, stream, a);
    cudaError_t e = launch_pdl(kv_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv_compact_move_kernel, dim3(148 * 4), dim3(kMoveThreads), 0, stream, a);
}

}  // namespace exl3
