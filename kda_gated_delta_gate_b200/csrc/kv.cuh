// Shared by the paged key-value cache calls (kda_kv.cu) and the attention over it (kda_attn_*.cu). Internal.
#pragma once

#include "common.cuh"

namespace kda {

// Host checks of a cache struct: sizes within the int arithmetic of the kernels, pools aligned.
inline int check_cache(const kda_kv_cache *c) {
    if (!c || !c->k || !c->v || !c->page_table || !c->seq_len || !c->ref) return KDA_ERR_INVALID_ARG;
    if (c->layers < 1 || c->num_pages < 1 || c->kv_heads < 1 || c->max_seqs < 1 || c->max_pages < 1)
        return KDA_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return KDA_ERR_UNSUPPORTED;
    const int ps = c->page_size;
    if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256) return KDA_ERR_UNSUPPORTED;
    // pool rows, table entries and positions are ints
    const long long rows = static_cast<long long>(c->num_pages) * c->kv_heads * ps;
    if (rows > 0x7fffffffLL || static_cast<long long>(c->num_pages) * c->kv_heads > 0x7fffffffLL / ps ||
        static_cast<long long>(c->max_pages) * ps > 0x7fffffffLL - 4096 ||
        static_cast<long long>(c->max_seqs) * c->max_pages > 0x7fffffffLL || c->kv_heads > 65535)
        return KDA_ERR_UNSUPPORTED;
    if (c->layers > 1 && c->layer_stride < rows * c->head_dim) return KDA_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v) || (c->layers > 1 && c->layer_stride % 8)) return KDA_ERR_MISALIGNED;
    return KDA_OK;
}

// The cache as the kernels see it; k and v at the layer of the call.
struct KvView {
    uint16_t *k, *v;
    int *table, *len, *ref;
    int num_pages, page_size, page_shift, kv_heads, max_seqs, max_pages;
};

inline KvView kv_view(const kda_kv_cache *c, int layer) {
    KvView w;
    w.k = c->k + static_cast<long long>(layer) * c->layer_stride;
    w.v = c->v + static_cast<long long>(layer) * c->layer_stride;
    w.table = c->page_table;
    w.len = c->seq_len;
    w.ref = c->ref;
    w.num_pages = c->num_pages;
    w.page_size = c->page_size;
    w.page_shift = __builtin_ctz(static_cast<unsigned>(c->page_size));
    w.kv_heads = c->kv_heads;
    w.max_seqs = c->max_seqs;
    w.max_pages = c->max_pages;
    return w;
}

// Programmatic dependent launch: let the next grid start; wait until the grids before have completed.
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_acquire() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch `kernel` so that it may start while the grid before it on the stream still runs (it waits in grid_acquire).
template <typename... P, typename... A>
int launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// Attention of a few query rows per sequence, split evenly over the cached rows on mma.sync (kda_attn_decode.cu): K rows
// of each sequence, or with cu (device, row bounds) at most K; few_rows(K, ..) holds.
size_t attn_rows_scratch_bytes(int K, int heads, const kda_kv_cache *cache);
int attn_rows(const kda_kv_cache *cache, int layer, const uint16_t *q, const int *cu, const int *slots, int N, int K,
              int total, int window, int sinks, uint16_t *out, float *lse, void *scratch, const kda_dims *dims,
              cudaStream_t s);
// The same in tiles of query rows on tcgen05 (kda_attn_prefill.cu): max_rows rows of each sequence, or with cu at most
// that many. attn_tiles_fits: the tiles' numbers are ints.
bool attn_tiles_fits(int B, int total, int heads, const kda_kv_cache *cache);
size_t attn_tiles_scratch_bytes(int B, int total, int heads, const kda_kv_cache *cache);
int attn_tiles(const kda_kv_cache *cache, int layer, const uint16_t *q, const int *cu, const int *slots, int B,
               int max_rows, int total, int window, int sinks, uint16_t *out, float *lse, void *scratch,
               const kda_dims *dims, cudaStream_t s);

// Up to 32 query rows per kv head take the split form, more the tiled one. 64 sequences of 4000 tokens, 8 kv heads of 128,
// 16 / 32 rows: 168 / 210 us split, 210 / 211 us tiled; 16 sequences of 500 to 8000 tokens, 32 rows: 75 split, 100 tiled (its
// CTAs take whole walks where they are many). 48 and 64 rows: 297 and 306 us with the split form taken that far, 211 and 213 tiled.
// (All tiled figures before its second sum of weights, which took 64 rows from 213 to 221.)
inline bool few_rows(int rows, int heads, const kda_kv_cache *cache) {
    return static_cast<long long>(heads / cache->kv_heads) * rows <= 32;
}

inline int check_scratch(const void *scratch, size_t bytes, size_t need) {
    if (!need) return KDA_OK;
    if (!scratch) return KDA_ERR_INVALID_ARG;
    if (!aligned16(scratch)) return KDA_ERR_MISALIGNED;
    return bytes < need ? KDA_ERR_CAPACITY : KDA_OK;
}

}  // namespace kda
