// exl3_cache.h -- launchers of the 4-bit products, the paged cache and the
// attention over it, shared between their translation units and api.cu.
#pragma once
#include "exl3_internal.h"

namespace exl3 {

// A launch that may begin while the previous kernel of its stream still runs
// (programmatic dependent launch): the kernel calls grid_dep_wait() before it
// touches memory.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// Products with plain 4-bit weights (q4.cu).
size_t q4_workspace_need(int m, int k_in, int n_out, int group);
size_t q4_workspace_bytes(int m, int k_in, int n_out);        // for up to m rows, whatever the groups
cudaError_t launch_q4_gemm(int m, const uint16_t* x, const uint32_t* packed, const uint16_t* scale,
                           const uint8_t* zero, void* y, int y_fp32, int k_in, int n_out, int group,
                           unsigned char* ws, cudaStream_t stream);
// The same for more rows (q4_tc.cu).
size_t q4_tc_workspace_bytes(int m, int k_in, int n_out);
cudaError_t launch_q4_tc(int m, const uint16_t* x, const uint32_t* packed, const uint16_t* scale, const uint8_t* zero,
                         void* y, int y_fp32, int k_in, int n_out, int group, unsigned char* ws, cudaStream_t stream);
cudaError_t launch_q4_pack(const uint8_t* q, int k_in, int n_out, uint32_t* packed, cudaStream_t stream);

// Paged key-value cache (kv_cache.cu) and the attention over it
// (paged_attn.cu).  The fault word and the call counters lie in front of the
// lists in the scratch memory (int32 words).
constexpr int kKvFault = 0;           // word: kKvFull | kKvIndex
constexpr int kKvArrived = 1;         // word: CTAs of an extend that are done
constexpr int kKvMoves = 2;           // word: pages a compaction moves
constexpr int kKvUsed = 3;            // word: used pages
constexpr int kKvLists = 64;          // n_pages words: sources, then destinations, of moves
constexpr int kKvMaxList = 1024;      // entries of a list of sequences
constexpr int kKvFull = 1, kKvIndex = 2;

struct KvArgs {
    uint16_t* k;
    uint16_t* v;
    int* table;
    int* lens;
    int* refs;
    uint32_t* free;
    int* scratch;
    int n_layers, n_pages, n_heads, page_size, head_dim, n_seqs, max_pages;
};

inline size_t kv_scratch_bytes(int n_pages)
{
    return sizeof(int) * ((size_t)kKvLists + (size_t)((n_pages + 63) / 64 * 64));
}
cudaError_t launch_kv_reset(const KvArgs& a, cudaStream_t stream);
cudaError_t launch_kv_extend(const KvArgs& a, int n, int m, const int* seqs, const int* counts, cudaStream_t stream);
cudaError_t launch_kv_write(const KvArgs& a, int layer, int n, int m, const int* seqs, const int* counts,
                            const uint16_t* k_new, const uint16_t* v_new, long long batch_stride,
                            long long row_stride, cudaStream_t stream);
cudaError_t launch_kv_truncate(const KvArgs& a, int n, const int* seqs, const int* new_lens, cudaStream_t stream);
cudaError_t launch_kv_fork(const KvArgs& a, int n, const int* src, const int* dst, cudaStream_t stream);
cudaError_t launch_kv_compact(const KvArgs& a, cudaStream_t stream);

struct AttnArgs {
    KvArgs c;
    int layer, n, m;
    const int* seqs;
    const int* counts;
    const uint16_t* q;
    long long q_bs, q_rs;
    int n_q_heads, group;             // group: query heads per head of the cache
    float scale;
    int window, sinks;
    uint16_t* out;
    long long o_bs, o_rs;
    float* lse;
    unsigned char* ws;
};
size_t attention_workspace_bytes(int m, int n_q_heads, int n_heads, int head_dim);
bool attention_tiles_ok(const AttnArgs& a);   // tiles are counted in 32 bits
int attention_launches(const KvArgs& c, int n, int m, int group);
cudaError_t launch_paged_attention(const AttnArgs& a, cudaStream_t stream);

}  // namespace exl3
