// The paged key-value cache (include/kda.h, kda_kv_cache): page bookkeeping on the device
// (reserve, fork, truncate, compact) and the writing of new rows (append).
//
// Bookkeeping is integer work over small arrays whose results feed each other (which pages are
// free, who gets which), so one block of 1024 threads does it with block-wide prefix sums and
// nothing reaches the host; what bounds it is the latency of a handful of dependent reads, not
// bytes. Rows that have to move (copies of partly filled pages, compaction) are listed in the
// cache's scratch and moved by a second, grid-wide launch that HBM bounds; it starts
// programmatically, so its launch overlaps the bookkeeping.
// Pages are given out lowest index first, in list order; atomics only add integers, so every
// result is the same on every run.
#include <algorithm>
#include <climits>

#include "kv.cuh"

namespace kda {
namespace {

constexpr int kBookThreads = 1024;

// The cache's scratch as int arrays. head[0]: entries of the copy list; head[1]: live pages (compaction).
struct BookScratch {
    int *head, *mark, *first, *len, *cow, *src, *dst, *rows, *map;
};
__host__ __device__ inline BookScratch book_scratch(int *p, int num_pages, int max_seqs) {
    BookScratch b;
    b.head = p;
    b.mark = p + 8;                 // per slot: the first listing of it
    b.first = b.mark + max_seqs;    // per pair: where its pages start in the list of taken ones, -1: refused
    b.len = b.first + max_seqs;     // per pair: length at the call's start (fork: the parent's)
    b.cow = b.len + max_seqs;       // per pair: 1 if its last page is shared and has to be copied
    b.src = b.cow + max_seqs;       // the copy list: page, page, filled rows
    b.dst = b.src + num_pages;
    b.rows = b.dst + num_pages;
    b.map = b.rows + num_pages;     // taken pages (lowest first), or new index per page (compaction)
    return b;
}
size_t book_scratch_ints(int num_pages, int max_seqs) {
    return 8 + 4 * static_cast<size_t>(max_seqs) + 4 * static_cast<size_t>(num_pages);
}

// Exclusive prefix sum of v over the block; total receives the sum. `sh` holds 32 values.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T &total, T *sh) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sh[w] = x;
    __syncthreads();
    if (w == 0) {
        T y = lane < nw ? sh[lane] : T(0);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        sh[lane] = y;
    }
    __syncthreads();
    const T base = w ? sh[w - 1] : T(0);
    total = sh[nw - 1];
    __syncthreads();
    return base + x - v;
}

// Calls visit(page, rank) for every page in [lo, hi) whose ref is 0 (WANT_FREE) or not, in index
// order by rank, until `want` have been found; returns how many there are (at most `want`). The whole
// block takes part; 4096 entries a round, the next ones requested while these are counted.
template <bool WANT_FREE, typename F>
__device__ int visit_pages(const int *ref, int lo, int hi, int want, int *sh, F visit) {
    const int t = threadIdx.x;
    int found = 0, r[4], next[4];
    auto fetch = [&](long long base, int (&x)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long p = base + 4 * t + j;
            x[j] = p < hi ? ref[p] : (WANT_FREE ? 1 : 0);
        }
    };
    fetch(lo, r);
    for (long long base = lo; base < hi && found < want; base += 4 * kBookThreads) {
        fetch(base + 4 * kBookThreads, next);
        int hit[4], sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hit[j] = (r[j] > 0) != WANT_FREE;
            sum += hit[j];
        }
        int total;
        int at = found + block_scan(sum, total, sh);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (hit[j] && at < want) visit(static_cast<int>(base) + 4 * t + j, at);
            at += hit[j];
            r[j] = next[j];
        }
        found += total;
    }
    __syncthreads();
    return min(found, want);
}

__device__ __forceinline__ int pages_of(int len, const KvView &c) {
    return (len >> c.page_shift) + ((len & (c.page_size - 1)) ? 1 : 0);
}
__device__ __forceinline__ bool is_page(int p, const KvView &c) { return p >= 0 && p < c.num_pages; }

// Reserve (from = null, add given) and fork (from = the parents, add = null).
template <bool FORK>
__global__ void __launch_bounds__(kBookThreads) take_pages_kernel(const KvView c, const int *__restrict__ from,
                                                                  const int *__restrict__ slots,
                                                                  const int *__restrict__ add, int n, int *scratch,
                                                                  int *status) {
    __shared__ long long shl[32];
    __shared__ int sh[32], bad, copies;
    grid_release();
    const BookScratch b = book_scratch(scratch, c.num_pages, c.max_seqs);
    const int tid = threadIdx.x;
    int *const taken = b.map;
    if (tid == 0) bad = 0, copies = 0;
    if (slots) {  // of several listings of a slot the first counts
        for (int i = tid; i < n; i += kBookThreads)
            if (slots[i] >= 0 && slots[i] < c.max_seqs) b.mark[slots[i]] = INT_MAX;
        __syncthreads();
        for (int i = tid; i < n; i += kBookThreads)
            if (slots[i] >= 0 && slots[i] < c.max_seqs) atomicMin(&b.mark[slots[i]], i);
    }
    __syncthreads();

    // what each pair needs, and where its pages lie in the list of taken ones
    long long base = 0;
    for (int i0 = 0; i0 < n; i0 += kBookThreads) {
        const int i = i0 + tid;
        int need = 0, cow = 0, len = 0;
        bool ok = false;
        if (i < n) {
            const int s = slots ? slots[i] : i;
            ok = s >= 0 && s < c.max_seqs && (!slots || b.mark[s] == i);
            if (FORK) {
                const int p = from[i];
                ok = ok && p >= 0 && p < c.max_seqs && p != s && c.len[s] == 0;
                len = ok ? c.len[p] : 0;
                ok = ok && len >= 0 && len <= c.max_pages * c.page_size;
                const int rest = len & (c.page_size - 1);
                if (ok && rest) {
                    ok = is_page(c.table[static_cast<size_t>(p) * c.max_pages + (len >> c.page_shift)], c);
                    need = ok ? 1 : 0;
                }
            } else {
                const int a = add[i];
                len = ok ? c.len[s] : 0;
                ok = ok && a >= 0 && len >= 0 &&
                     static_cast<long long>(len) + a <= static_cast<long long>(c.max_pages) * c.page_size;
                if (ok && a > 0 && (len & (c.page_size - 1))) {
                    const int last = c.table[static_cast<size_t>(s) * c.max_pages + (len >> c.page_shift)];
                    ok = is_page(last, c);
                    cow = ok && c.ref[last] > 1;
                }
                need = ok ? pages_of(len + a, c) - pages_of(len, c) + cow : 0;
            }
            if (!ok) bad = KDA_ERR_INVALID_ARG;
        }
        long long total;
        const long long at = base + block_scan<long long>(need, total, shl);
        if (i < n) {
            b.first[i] = ok ? static_cast<int>(min(at, static_cast<long long>(c.num_pages))) : -1;
            b.len[i] = len;
            b.cow[i] = cow;
        }
        base += total;
    }
    __syncthreads();
    int have = 0;
    if (base > 0)
        have = visit_pages<true>(c.ref, 0, c.num_pages, static_cast<int>(min(base, static_cast<long long>(c.num_pages))),
                                 sh, [&](int page, int rank) { taken[rank] = page; });

    // `wide` threads per pair, so that few pairs of many pages and many pairs of few both take few rounds; refs and
    // lengths have all been read by now
    int wide = kBookThreads;
    while (wide > 4 && n > kBookThreads / wide) wide >>= 1;
    const int lane = tid & (wide - 1);
    for (int i = tid / wide; i < n; i += kBookThreads / wide) {
        int first = b.first[i];
        if (first < 0) continue;
        const int s = slots ? slots[i] : i, len = b.len[i];
        int *const row = c.table + static_cast<size_t>(s) * c.max_pages;
        const int rest = len & (c.page_size - 1), full = len >> c.page_shift;
        const int cow = FORK ? (rest ? 1 : 0) : b.cow[i];
        const int p0 = pages_of(len, c), more = FORK ? 0 : pages_of(len + add[i], c) - p0;
        if (more + cow > have - first && more + cow > 0) {
            if (lane == 0) bad = KDA_ERR_CAPACITY;
            continue;
        }
        const int *const prow = FORK ? c.table + static_cast<size_t>(from[i]) * c.max_pages : row;
        if (FORK)
            for (int j = lane; j < full; j += wide) {
                const int pg = prow[j];
                row[j] = pg;
                if (is_page(pg, c)) atomicAdd(&c.ref[pg], 1);
            }
        if (cow) {  // the partly filled last page: a page of its own, the filled rows copied
            if (lane == 0) {
                const int pg = taken[first], src = prow[full], e = atomicAdd(&copies, 1);
                b.src[e] = src;
                b.dst[e] = pg;
                b.rows[e] = rest;
                row[full] = pg;
                c.ref[pg] = 1;
                if (!FORK) atomicSub(&c.ref[src], 1);
            }
            ++first;
        }
        for (int j = lane; j < more; j += wide) {
            const int pg = taken[first + j];
            row[p0 + j] = pg;
            c.ref[pg] = 1;
        }
        if (lane == 0) c.len[s] = FORK ? len : len + add[i];
    }
    __syncthreads();
    if (tid == 0) {
        b.head[0] = copies;
        if (bad) atomicExch(status, bad);
    }
}

// One block per listed slot: the pages past the kept tokens leave the table row.
__global__ void __launch_bounds__(128) truncate_kernel(const KvView c, const int *__restrict__ slots,
                                                       const int *__restrict__ new_len, int n, int *status) {
    const int i = blockIdx.x, tid = threadIdx.x;
    const int s = slots ? slots[i] : i, keep = new_len[i];
    int twice = 0;
    if (slots)
        for (int j = tid; j < i; j += blockDim.x) twice |= slots[j] == s;
    const bool in = s >= 0 && s < c.max_seqs;
    const int len = in ? c.len[s] : 0;  // read before the barrier, written after it by this block alone
    twice = __syncthreads_or(twice);
    if (!in || twice || keep < 0 || keep > len || len > c.max_pages * c.page_size) {
        if (tid == 0) atomicExch(status, KDA_ERR_INVALID_ARG);
        return;
    }
    int *const row = c.table + static_cast<size_t>(s) * c.max_pages;
    for (int j = pages_of(keep, c) + tid; j < pages_of(len, c); j += blockDim.x) {
        const int pg = row[j];
        if (is_page(pg, c)) atomicSub(&c.ref[pg], 1);
        row[j] = -1;
    }
    if (tid == 0) c.len[s] = keep;
}

// The moves of a compaction: L live pages; the i-th live page at or past L goes to the i-th free one below L.
__global__ void __launch_bounds__(kBookThreads) compact_plan_kernel(const KvView c, int *scratch, int *live_out) {
    __shared__ int sh[32];
    grid_release();
    const BookScratch b = book_scratch(scratch, c.num_pages, c.max_seqs);
    const int tid = threadIdx.x;
    int mine = 0;
    for (int p = tid; p < c.num_pages; p += kBookThreads) mine += c.ref[p] > 0;
    int live;
    block_scan(mine, live, sh);
    for (int p = live + tid; p < c.num_pages; p += kBookThreads) b.map[p] = p;
    __syncthreads();
    const int holes = visit_pages<true>(c.ref, 0, live, INT_MAX, sh, [&](int page, int rank) { b.dst[rank] = page; });
    visit_pages<false>(c.ref, live, c.num_pages, holes, sh, [&](int page, int rank) { b.src[rank] = page; });
    for (int i = tid; i < holes; i += kBookThreads) {
        const int src = b.src[i], dst = b.dst[i];
        b.rows[i] = c.page_size;
        b.map[src] = dst;
        c.ref[dst] = c.ref[src];
        c.ref[src] = 0;
    }
    if (tid == 0) {
        b.head[0] = holes;
        b.head[1] = live;
        if (live_out) *live_out = live;
    }
}

// The listed page copies in every layer and both pools, and (REMAP) the table's entries at or past the
// live count. A (page, head) block is contiguous; a warp moves 2 KB of it at a time, four 16-byte
// loads in flight per lane, so that eight 256-thread blocks keep 128 KB per SM moving. Measured: 2048 pages of 64 rows,
// 8 heads of 128, 4 layers (2.1 GB read and written) in 331 us = 6.5 TB/s, the card's copy rate.
constexpr int kCopyThreads = 256, kPieceBytes = 2048;
template <bool REMAP>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(uint16_t *k, uint16_t *v, long long layer_stride,
                                                                  int layers, const KvView c, int head_dim,
                                                                  int *scratch) {
    grid_acquire();
    const BookScratch b = book_scratch(scratch, c.num_pages, c.max_seqs);
    const int lane = threadIdx.x & 31;
    const int row_bytes = head_dim * 2, block_bytes = c.page_size * row_bytes, pieces = block_bytes / kPieceBytes;
    const long long per_entry = 2LL * layers * c.kv_heads * pieces;
    const long long total = per_entry * b.head[0];
    const long long step = static_cast<long long>(gridDim.x) * (kCopyThreads / 32);
    for (long long u = static_cast<long long>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5); u < total; u += step) {
        const int e = static_cast<int>(u / per_entry);
        int r = static_cast<int>(u - e * per_entry);
        const int piece = r % pieces;
        r /= pieces;
        const int h = r % c.kv_heads;
        r /= c.kv_heads;
        uint16_t *const pool = (r & 1 ? v : k) + static_cast<long long>(r >> 1) * layer_stride;
        const int bytes = b.rows[e] * row_bytes - piece * kPieceBytes;  // of this piece that are filled
        const size_t off = static_cast<size_t>(piece) * kPieceBytes + 16 * lane;
        const char *src = reinterpret_cast<const char *>(pool) +
                          (static_cast<size_t>(b.src[e]) * c.kv_heads + h) * block_bytes + off;
        char *dst = reinterpret_cast<char *>(pool) + (static_cast<size_t>(b.dst[e]) * c.kv_heads + h) * block_bytes + off;
        uint4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (512 * j + 16 * lane < bytes) x[j] = __ldcs(reinterpret_cast<const uint4 *>(src + 512 * j));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (512 * j + 16 * lane < bytes) __stcs(reinterpret_cast<uint4 *>(dst + 512 * j), x[j]);
    }
    if (REMAP) {
        const int live = b.head[1];
        const long long entries = static_cast<long long>(c.max_seqs) * c.max_pages;
        for (long long i = blockIdx.x * static_cast<long long>(kCopyThreads) + threadIdx.x; i < entries;
             i += static_cast<long long>(gridDim.x) * kCopyThreads) {
            const int p = c.table[i];
            if (p >= live && p < c.num_pages) c.table[i] = b.map[p];
        }
    }
}

// New rows into their pages. A block takes R consecutive rows. Its threads first request their first 16-byte pieces
// (K and V rows of kv_heads * head_dim values are contiguous on the way in, head_dim values on the way out), then find
// the rows' places (four dependent reads, which those loads cover), then store and go on, kPieces at a time.
// R grows with the rows so that small calls still spread over the SMs. 36.9 K rows of 8 heads of 128: 57.6 us (5.2 TB/s read and
// written) with four pieces in flight per thread, 59.8 with eight and 84.8 with sixteen (fewer blocks fit an SM).
constexpr int kAppendThreads = 256, kAppendRows = 16, kPieces = 4;
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const KvView c, int head_dim,
                                                                const uint16_t *__restrict__ k_new,
                                                                const uint16_t *__restrict__ v_new, long long ld,
                                                                const int *__restrict__ cu,
                                                                const int *__restrict__ slots, int B, int total, int R,
                                                                int *status) {
    __shared__ long long place[kAppendRows];  // element offset of (page, head 0, row) in the pools, or -1
    __shared__ int seq[kAppendRows], twice[kAppendRows];
    const int tid = threadIdx.x, row0 = blockIdx.x * R, rows = min(R, total - row0);
    if (tid < kAppendRows) {
        seq[tid] = INT_MAX;
        twice[tid] = 0;
    }
    __syncthreads();
    const int end = cu[B];  // rows behind the last sequence may be anything, unmapped included
    const int per_head = head_dim / 8, per_row = c.kv_heads * per_head, pieces = rows * 2 * per_row;
    uint4 x[kPieces];
    auto request = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int i = i0 + j * kAppendThreads, r = i / (2 * per_row);
            if (i < pieces && row0 + r < end) {
                const int w = i - r * 2 * per_row, kv = w >= per_row, e = kv ? w - per_row : w;
                x[j] = __ldg(reinterpret_cast<const uint4 *>((kv ? v_new : k_new) + (row0 + r) * ld + 8 * e));
            }
        }
    };
    request(tid);
    // the sequence of every row: thread b marks its own; beyond a few rounds of that, a bisection per row
    auto bounds = [&](int b, int &c0, int &c1) {
        c0 = cu[b];
        c1 = cu[b + 1];
        return c0 >= 0 && c1 >= c0 && c1 <= total && c1 <= end;
    };
    int c0, c1;
    for (int b = blockIdx.x * kAppendThreads + tid; b < B; b += gridDim.x * kAppendThreads)
        if (!bounds(b, c0, c1)) atomicExch(status, KDA_ERR_INVALID_ARG);
    if (B <= 4 * kAppendThreads) {
        for (int b = tid; b < B; b += kAppendThreads)
            if (bounds(b, c0, c1))
                for (int r = max(c0 - row0, 0); r < min(c1 - row0, rows); ++r) atomicMin(&seq[r], b);
    } else if (tid < rows && row0 + tid < end) {
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= row0 + tid) lo = mid;
            else hi = mid;
        }
        if (bounds(lo, c0, c1) && c0 <= row0 + tid && row0 + tid < c1) seq[tid] = lo;
    }
    __syncthreads();
    if (tid < rows) {
        const int b = seq[tid];
        long long to = -1;
        if (b < B) {
            const int s = slots ? slots[b] : b;
            const int c0 = cu[b], n = cu[b + 1] - c0, t = row0 + tid - c0;
            bool bad = true;
            if (s >= 0 && s < c.max_seqs) {
                const int len = c.len[s], at = len - n + t;
                if (len <= c.max_pages * c.page_size && len >= n) {
                    const int pg = c.table[static_cast<size_t>(s) * c.max_pages + (at >> c.page_shift)];
                    if (is_page(pg, c) && c.ref[pg] == 1) {
                        bad = false;
                        to = (static_cast<long long>(pg) * c.kv_heads * c.page_size + (at & (c.page_size - 1))) * head_dim;
                    }
                }
            }
            if (bad) atomicExch(status, KDA_ERR_INVALID_ARG);
        }
        place[tid] = to;
    }
    if (slots) {  // a slot listed before: its first listing's rows count
        for (int r = 0; r < rows; ++r) {
            const int b = seq[r];
            if (b >= B || (r && seq[r - 1] == b)) continue;  // the first row of each sequence in the block
            const int s = slots[b];
            for (int j = tid; j < b; j += kAppendThreads)
                if (slots[j] == s) twice[r] = 1;
        }
        __syncthreads();
        if (tid < rows && seq[tid] < B) {
            int r = tid;
            while (r && seq[r - 1] == seq[tid]) --r;
            if (twice[r]) {
                place[tid] = -1;
                atomicExch(status, KDA_ERR_INVALID_ARG);
            }
        }
    }
    __syncthreads();
    const long long head_step = static_cast<long long>(c.page_size) * head_dim;
    for (int i0 = tid; i0 < pieces; i0 += kPieces * kAppendThreads) {
        if (i0 != tid) request(i0);
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int i = i0 + j * kAppendThreads;
            if (i >= pieces) break;
            const int r = i / (2 * per_row), w = i - r * 2 * per_row, kv = w >= per_row, e = kv ? w - per_row : w;
            if (place[r] >= 0)
                *reinterpret_cast<uint4 *>((kv ? c.v : c.k) + place[r] + (e / per_head) * head_step + 8 * (e % per_head)) = x[j];
        }
    }
}

int check_book(const kda_kv_cache *c) {
    KDA_TRY(check_cache(c));
    if (!c->scratch) return KDA_ERR_INVALID_ARG;
    if (!aligned16(c->scratch)) return KDA_ERR_MISALIGNED;
    return KDA_OK;
}

// Blocks for at most `entries` page copies of the cache.
int copy_grid(const kda_kv_cache *c, long long entries) {
    const long long pieces = entries * 2 * c->layers * c->kv_heads * (c->page_size * c->head_dim * 2 / kPieceBytes);
    return static_cast<int>(std::min<long long>(std::max<long long>((pieces + 7) / 8, 1), 8LL * num_sms()));
}

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_kv_scratch_bytes(int num_pages, int max_seqs) {
    if (num_pages < 1 || max_seqs < 1) return 0;
    return (kda::book_scratch_ints(num_pages, max_seqs) * sizeof(int) + 15) / 16 * 16;
}

int kda_kv_reserve(const kda_kv_cache *cache, const int *slots, const int *add, int n, void *stream) {
    KDA_TRY(kda::check_book(cache));
    if (!add || n < 0 || n > cache->max_seqs) return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    int *status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    auto s = static_cast<cudaStream_t>(stream);
    const kda::KvView view = kda::kv_view(cache, 0);
    kda::take_pages_kernel<false><<<1, kda::kBookThreads, 0, s>>>(view, nullptr, slots, add, n, cache->scratch, status);
    KDA_TRY(kda::launch_status());
    return kda::launch_after(kda::copy_pages_kernel<false>, dim3(kda::copy_grid(cache, n)), dim3(kda::kCopyThreads), 0, s,
                             cache->k, cache->v, cache->layer_stride, cache->layers, view, cache->head_dim,
                             cache->scratch);
}

int kda_kv_fork(const kda_kv_cache *cache, const int *parent, const int *child, int n, void *stream) {
    KDA_TRY(kda::check_book(cache));
    if (!parent || !child || n < 0 || n > cache->max_seqs) return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    int *status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    auto s = static_cast<cudaStream_t>(stream);
    const kda::KvView view = kda::kv_view(cache, 0);
    kda::take_pages_kernel<true><<<1, kda::kBookThreads, 0, s>>>(view, parent, child, nullptr, n, cache->scratch, status);
    KDA_TRY(kda::launch_status());
    return kda::launch_after(kda::copy_pages_kernel<false>, dim3(kda::copy_grid(cache, n)), dim3(kda::kCopyThreads), 0, s,
                             cache->k, cache->v, cache->layer_stride, cache->layers, view, cache->head_dim,
                             cache->scratch);
}

int kda_kv_truncate(const kda_kv_cache *cache, const int *slots, const int *new_len, int n, void *stream) {
    KDA_TRY(kda::check_cache(cache));
    if (!new_len || n < 0 || n > cache->max_seqs) return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    int *status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    kda::truncate_kernel<<<n, 128, 0, static_cast<cudaStream_t>(stream)>>>(kda::kv_view(cache, 0), slots, new_len, n,
                                                                          status);
    return kda::launch_status();
}

int kda_kv_compact(const kda_kv_cache *cache, int *live, void *stream) {
    KDA_TRY(kda::check_book(cache));
    auto s = static_cast<cudaStream_t>(stream);
    const kda::KvView view = kda::kv_view(cache, 0);
    kda::compact_plan_kernel<<<1, kda::kBookThreads, 0, s>>>(view, cache->scratch, live);
    KDA_TRY(kda::launch_status());
    return kda::launch_after(kda::copy_pages_kernel<true>, dim3(kda::copy_grid(cache, cache->num_pages / 2 + 1)),
                             dim3(kda::kCopyThreads), 0, s, cache->k, cache->v, cache->layer_stride, cache->layers, view,
                             cache->head_dim, cache->scratch);
}

int kda_kv_append(const kda_kv_cache *cache, int layer, const kda_bf16 *k_new, const kda_bf16 *v_new, long long ld,
                  const int *cu_seqlens, const int *slots, int B, int total_tokens, void *stream) {
    KDA_TRY(kda::check_cache(cache));
    if (!k_new || !v_new || !cu_seqlens || B < 0 || total_tokens < 0 || layer < 0 || layer >= cache->layers)
        return KDA_ERR_INVALID_ARG;
    if (ld < static_cast<long long>(cache->kv_heads) * cache->head_dim) return KDA_ERR_INVALID_ARG;
    if (!kda::aligned16(k_new) || !kda::aligned16(v_new) || ld % 8) return KDA_ERR_MISALIGNED;
    if (static_cast<long long>(cache->kv_heads) * cache->head_dim > (1 << 20)) return KDA_ERR_UNSUPPORTED;
    if (B == 0 || total_tokens == 0) return KDA_OK;
    int *status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    const int R = std::min(kda::kAppendRows, std::max(1, total_tokens / (4 * kda::num_sms())));
    kda::append_kernel<<<(total_tokens + R - 1) / R, kda::kAppendThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        kda::kv_view(cache, layer), cache->head_dim, k_new, v_new, ld, cu_seqlens, slots, B, total_tokens, R, status);
    return kda::launch_status();
}

}  // extern "C"
