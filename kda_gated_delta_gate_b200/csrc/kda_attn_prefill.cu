// Attention of packed query rows over their paged cache (include/kda.h, kda_attn_prefill).
#include "kv.cuh"

namespace kda {
namespace {

// One warp per (row, head): an online softmax over the visible rows, lanes along the channels.
template <int D>
__global__ void __launch_bounds__(128) prefill_kernel(const KvView c, const uint16_t *q, const int *cu, const int *slots,
                                                      int B, int max_rows, int total, int heads, int window, int sinks,
                                                      float scale, uint16_t *out, float *lse, int *status) {
    constexpr int E = D / 32;
    const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
    const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
    const int c0 = cu[b], c1 = cu[b + 1], s = slots ? slots[b] : b, n = c1 - c0;
    int len = 0;
    bool ok = c0 >= 0 && c1 >= c0 && c1 <= total && n <= max_rows && s >= 0 && s < c.max_seqs;
    if (ok) len = c.len[s];
    ok = ok && len >= 0 && len <= c.max_pages * c.page_size;
    if (!ok) {
        if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) atomicExch(status, KDA_ERR_INVALID_ARG);
        return;
    }
    if (t >= n) return;
    const int p = len - n + t, hkv = h / (heads / c.kv_heads);
    const size_t row = static_cast<size_t>(c0 + t) * heads + h;
    float qv[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) qv[e] = bf16_to_f32(q[row * D + lane + 32 * e]), o[e] = 0.f;
    const int lo = window ? max(0, p - window + 1) : 0;
    for (int j = (lo > 0 && sinks > 0) ? 0 : lo; j <= p; ++j) {
        if (j < lo && j >= sinks) { j = lo - 1; continue; }
        const int pg = c.table[static_cast<size_t>(s) * c.max_pages + (j >> c.page_shift)];
        if (pg < 0 || pg >= c.num_pages) {
            if (lane == 0) atomicExch(status, KDA_ERR_INVALID_ARG);
            return;
        }
        const size_t off = ((static_cast<size_t>(pg) * c.kv_heads + hkv) * c.page_size + (j & (c.page_size - 1))) * D + lane;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x = fmaf(qv[e], bf16_to_f32(c.k[off + 32 * e]), x);
#pragma unroll
        for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
        x *= scale;
        const float mn = fmaxf(m, x), f = expf(m - mn), w = expf(x - mn);
        m = mn;
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * bf16_to_f32(c.v[off + 32 * e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) out[row * D + lane + 32 * e] = f32_to_bf16(l == 0.f ? 0.f : o[e] / l);
    if (lse && lane == 0) lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace
}  // namespace kda

extern "C" int kda_attn_prefill(const kda_kv_cache *cache, int layer, const kda_bf16 *q, const int *cu_seqlens,
                                const int *slots, int B, int max_rows, int total_tokens, int window, int sinks,
                                kda_bf16 *out, float *lse, const kda_dims *dims, void *stream) {
    KDA_TRY(kda::check_cache(cache));
    KDA_TRY(kda::check_dims(dims));
    if (!q || !cu_seqlens || !out || B < 0 || max_rows < 0 || total_tokens < 0 || window < 0 || sinks < 0 || layer < 0 ||
        layer >= cache->layers)
        return KDA_ERR_INVALID_ARG;
    if (dims->head_dim != cache->head_dim || dims->heads % cache->kv_heads) return KDA_ERR_INVALID_ARG;
    if (!kda::aligned16(q) || !kda::aligned16(out)) return KDA_ERR_MISALIGNED;
    if (B > 65535 || dims->heads > 65535) return KDA_ERR_UNSUPPORTED;
    if (B == 0 || total_tokens == 0) return KDA_OK;
    if (max_rows == 0) return KDA_ERR_INVALID_ARG;
    int *status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    const dim3 grid((max_rows + 3) / 4, dims->heads, B);
    auto s = static_cast<cudaStream_t>(stream);
    const kda::KvView view = kda::kv_view(cache, layer);
    if (dims->head_dim == 128)
        kda::prefill_kernel<128><<<grid, 128, 0, s>>>(view, q, cu_seqlens, slots, B, max_rows, total_tokens, dims->heads,
                                                     window, sinks, dims->scale, out, lse, status);
    else
        kda::prefill_kernel<64><<<grid, 128, 0, s>>>(view, q, cu_seqlens, slots, B, max_rows, total_tokens, dims->heads,
                                                    window, sinks, dims->scale, out, lse, status);
    return kda::launch_status();
}
