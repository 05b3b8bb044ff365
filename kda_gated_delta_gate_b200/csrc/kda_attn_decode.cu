// Attention of the last K tokens of N sequences over their paged cache (include/kda.h, kda_attn_decode).
//
// Per (sequence, kv head): S = scale q k^T over the visible rows, o = softmax(S) v, in one pass with
// the running maximum m and sum l of the softmax (base 2): p = 2^(s - m), l += sum p, o = o 2^(m_old - m) + p v.
// The G K query rows of a kv head (G query heads per kv head) share every K and V row read, so the pass
// moves 4 D bytes per cached row and head for 4 G K D flops: HBM bounds it.
//
// Split: the visible tiles (64 rows at head_dim 128, 128 at 64) of all (sequence, kv head) pairs form one list; each CTA
// of a fixed grid (the resident CTAs of the card) takes an equal run of it, whatever the mix of lengths. A pair that
// falls into one run is finished there; a pair that runs cut leaves (m, l, o) per CTA in scratch, and
// join_kernel adds the parts in a fixed order (the same bits on every call).
//
// A CTA is four warps over one tile: K and V rows arrive by 16-byte cp.async, one or two tiles ahead, in shared memory whose
// 16-byte chunks are permuted by chunk ^ (row % 8); mma.sync (m16n8k16, BF16 in, FP32 sums) takes them by ldmatrix.
// With at most 16 query rows each warp takes a quarter of the tile's keys and its own m, l and o, joined at the pair's
// end; with up to 32 two warps share a key half. With at most 8 the products are turned round (RowsShort). mma.sync is
// enough: at 16 rows the products need about a sixth of its rate while HBM is saturated.
// p is rounded to BF16 for the second product (at most 2^-8 of each weight); the sum that o is divided by is that of the
// rounded p (one more product, with ones), so that the roundings cancel where few keys carry a row, and the one that
// lse takes is that of the unrounded p.
//
// Measured (6545 GB/s is a copy's rate; reads alone go a little faster). 8 x 65500 tokens, 8 kv heads of 128, 4 rows per kv
// head: 323 us = 6.6 TB/s in bursts of 20 on states in turn, 342 us = 6.3 TB/s in a loop, once the card is warm; 64 sequences of
// 125 to 8000 tokens: 4 rows 171 us = 6.2 TB/s (181 in a loop), 16 rows 209 us = 5.1 TB/s in a loop; at head_dim 64, 4 rows, 92 us =
// 5.8 TB/s. 256 sequences of 8000, window 1024, 4 sinks: 174 us = 6.2 TB/s, at head_dim 64 102 us = 5.3 TB/s. One sequence of 4096:
// 11.9 us (one state, replayed, so out of L2), nearly all of it the latency of two launches and of the reads that depend on
// one another (slot, length, table, K, parts).
#include <algorithm>
#include <type_traits>

#include "kv.cuh"

namespace kda {
namespace {

// Cached rows per tile: 32 KB of K and V at either head_dim (at 64, 64 ragged sequences of 125 to 8000 tokens, 8 kv heads, 533 MB:
// 104.6 us with 64 rows a tile and four stages, 91.2 with 128 and two)
__host__ __device__ constexpr int tile_of(int D) { return D == 64 ? 128 : 64; }
constexpr int kThreads = 128;  // four warps
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct DecodeArgs {
    KvView c;
    const uint16_t *q;
    const int *cu;  // row bounds of the sequences, or null: K rows each
    const int *slots;
    uint16_t *out;
    float *lse;
    float *part_o, *part_ml;  // [CTA][2][rows][D], [CTA][2][rows][4]: m, l (-1: bad page), l of the rounded p
    long long *info;          // [0] all tiles; then per CTA, of the pair that its run starts in: kv head, first tile in the
                              // list, tiles, first query row, query rows
    int *status;
    int N, K, G, heads, window, sinks;  // K: rows per sequence, with cu the most of any
    int total;                          // with cu: rows of q
    float scale2;  // scale * log2(e)
};

// The tiles of one sequence: `sink` leading ones, then those from `lo / 64` to the last.
struct Span {
    int len, lo, sink, tiles;  // tiles = 0: the sequence is skipped
    int row0, n;               // its query rows
};
// What a sequence's span is made of, read without branches so that several sequences' reads can be in flight.
struct Bounds {
    int c0, c1, slot, len;  // len -1: the slot is none
};
__device__ __forceinline__ Bounds bounds_of(const DecodeArgs &a, int n) {
    Bounds b;
    b.slot = a.slots ? a.slots[n] : n;
    b.c0 = a.cu ? a.cu[n] : n * a.K;
    b.c1 = a.cu ? a.cu[n + 1] : n * a.K + a.K;
    b.len = b.slot >= 0 && b.slot < a.c.max_seqs ? a.c.len[b.slot] : -1;
    return b;
}
template <int kTile>
__device__ __forceinline__ Span span_of(const DecodeArgs &a, const Bounds &b, bool &bad) {
    Span s{0, 0, 0, 0, b.c0, b.c1 - b.c0};
    bad = b.c0 < 0 || b.c1 < b.c0 || b.c1 > a.total || b.c1 - b.c0 > a.K || b.len < 0 || b.len > a.c.max_pages * a.c.page_size;
    if (bad || s.n == 0) return s;
    s.len = b.len;
    s.lo = a.window ? max(0, b.len - s.n - a.window + 1) : 0;
    if (s.lo > 0) s.sink = min((min(a.sinks, s.lo) + kTile - 1) / kTile, s.lo / kTile);
    s.tiles = max(1, s.sink + (b.len + kTile - 1) / kTile - s.lo / kTile);  // an empty one still writes its zeros
    return s;
}
template <int kTile>
__device__ __forceinline__ int tile_row0(const Span &s, int i) {
    return (i < s.sink ? i : i - s.sink + s.lo / kTile) * kTile;
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool fill) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// An 8 x 8 matrix of 16-bit values, a row's two neighbours per thread, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
constexpr uint32_t kOnes = 0x3f803f80u;  // two BF16 ones
// The score in base 2 of cached row j for a row at position p; -inf where it is hidden.
__device__ __forceinline__ float seen_score(const DecodeArgs &a, float s, bool all_seen, int j, int p) {
    s *= a.scale2;
    if (all_seen) return s;
    return j <= p && (!a.window || j > p - a.window || j < a.sinks) ? s : -INFINITY;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// Tile runs: CTA c of `ctas` (below 1024) takes tiles [run_start(c), run_start(c + 1)).
__device__ __forceinline__ long long run_start(long long tiles, int ctas, int c) {
    if (tiles < (1 << 22)) return static_cast<unsigned>(tiles) * static_cast<unsigned>(c) / static_cast<unsigned>(ctas);
    return tiles * c / ctas;
}
// The run that holds tile x: the last c with tiles c / ctas < x + 1.
__device__ __forceinline__ int run_of(long long tiles, int ctas, long long x) {
    return static_cast<int>(((x + 1) * ctas + tiles - 1) / tiles) - 1;
}

// A warp's share of a tile in the two forms. Both hold, for the warp's keys, the rows' queries, m, l, the sums lp of the
// rounded p and o, and have:
//   fetch   the rows' queries and positions (called before the last pair's results are written, so that the loads run
//           under that);  begin  an empty softmax;  tile  one tile;  put  m, l, lp to ml and o to the join buffer,
//           where channel d of row r lies at place(r, d): groups of eight channels are permuted so that what a warp writes
//           at once goes to different banks.

// Up to 8 rows: K q^T (keys x rows) and V^T p^T (channels x rows), rows on the products' short side, so that none is
// spent on padding to 16. Thread: rows 2 (lane % 4) + e. Against the other form (8 x 65500 tokens, 4 rows per kv head, replayed on
// one state): 315 us against 320, and 316 against 340 after some seconds, since it does half the products.
template <int D>
struct RowsShort {
    static constexpr int KG = 4, ROWS = 8, KPW = tile_of(D) / KG;
    uint32_t qf[D / 16][2];
    float o[D / 16][4], m[2], l[2], lp[4];
    int pos[2];
    static __device__ __forceinline__ int keys0(int warp) { return KPW * warp; }
    static __device__ __forceinline__ int place(int r, int d) { return r * D + (d ^ (((r >> 1) & 3) << 3)); }
    __device__ __forceinline__ void fetch(const DecodeArgs &a, const Span &sp, int h, int, int lane) {
        const int rows = a.G * sp.n, r = lane >> 2, t = r / a.G;
        const uint16_t *const q = a.q + (static_cast<size_t>(sp.row0 + t) * a.heads + static_cast<size_t>(h) * a.G + (r - t * a.G)) * D +
                                  2 * (lane & 3);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            qf[ks][0] = r < rows ? __ldg(reinterpret_cast<const uint32_t *>(q + 16 * ks)) : 0u;
            qf[ks][1] = r < rows ? __ldg(reinterpret_cast<const uint32_t *>(q + 16 * ks + 8)) : 0u;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) pos[e] = sp.len - sp.n + min((2 * (lane & 3) + e) / a.G, sp.n - 1);
    }
    __device__ __forceinline__ void begin() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
        lp[0] = lp[1] = lp[2] = lp[3] = 0.f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    }
    // j0: the warp's first key; all_seen: every row sees all of its keys
    __device__ __forceinline__ void tile(const DecodeArgs &a, uint32_t sk, uint32_t sv, int j0, bool all_seen, int warp, int lane) {
        float s[KPW / 16][4], top[2] = {-INFINITY, -INFINITY}, safe[2];
#pragma unroll
        for (int kb = 0; kb < KPW / 16; ++kb) {
            s[kb][0] = s[kb][1] = s[kb][2] = s[kb][3] = 0.f;
            // matrices: keys +0..7 / +8..15 (lane bit 3), channels +0..7 / +8..15 (lane bit 4)
            const int r = keys0(warp) + 16 * kb + (lane & 15);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t k[4];
                ldsm4(sk + r * D * 2 + (((2 * ks + (lane >> 4)) ^ (r & 7)) << 4), k);
                mma16816(s[kb], k, qf[ks][0], qf[ks][1]);
            }
        }
#pragma unroll
        for (int kb = 0; kb < KPW / 16; ++kb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[kb][e] = seen_score(a, s[kb][e], all_seen, j0 + 16 * kb + (lane >> 2) + 8 * (e >> 1), pos[e & 1]);
                top[e & 1] = fmaxf(top[e & 1], s[kb][e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], w));
            const float mn = fmaxf(m[e], top[e]);
            safe[e] = mn == -INFINITY ? 0.f : mn;
            const float f = ex2(m[e] - safe[e]);
            m[e] = mn;
            l[e] *= f;
            lp[e] *= f;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                o[d][e] *= f;
                o[d][2 + e] *= f;
            }
        }
#pragma unroll
        for (int kb = 0; kb < KPW / 16; ++kb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[kb][e] = ex2(s[kb][e] - safe[e & 1]);
                l[e & 1] += s[kb][e];
            }
        }
#pragma unroll
        for (int kb = 0; kb < KPW / 16; ++kb) {
            // p of 16 keys: from (key, two rows) to (row, two keys) per thread
            const uint32_t p0 = transpose8(pack_bf16(s[kb][0], s[kb][1])), p1 = transpose8(pack_bf16(s[kb][2], s[kb][3]));
            const uint32_t ones[4] = {kOnes, kOnes, kOnes, kOnes};
            mma16816(lp, ones, p0, p1);
            // matrices: keys +0..7 / +8..15 (lane bit 4), channels +0..7 / +8..15 (lane bit 3)
            const int r = keys0(warp) + 16 * kb + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                uint32_t v[4];
                ldsm4t(sv + r * D * 2 + (((2 * d + ((lane >> 3) & 1)) ^ (r & 7)) << 4), v);
                mma16816(o[d], v, p0, p1);
            }
        }
    }
    __device__ __forceinline__ void put_sums(float4 *ml, int warp, int lane) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], w);
            if (lane < 4) ml[warp * ROWS + 2 * lane + e] = make_float4(m[e], l[e], lp[e], 0.f);
        }
    }
    __device__ __forceinline__ void put_o(float *so, int rows, int warp, int lane) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 2 * (lane & 3) + (e & 1);
            if (r < rows) {
                float *const w = so + (warp * ROWS + r) * D + (lane >> 2);
#pragma unroll
                for (int d = 0; d < D / 16; ++d) w[8 * ((2 * d + (e >> 1)) ^ (lane & 3))] = o[d][e];
            }
        }
    }
};

// Up to 16 MT rows: q K^T (rows x keys) and p V (rows x channels). Thread: rows 16 (warp % MT) + lane / 4 and + 8; MT warps
// share a key group.
template <int D, int MT>
struct RowsLong {
    static constexpr int KG = 4 / MT, ROWS = 16 * MT, KPW = tile_of(D) / KG;
    uint32_t qf[D / 16][4];
    float o[D / 8][4], m[2], l[2], lp[4];
    int pos[2];
    static __device__ __forceinline__ int keys0(int warp) { return KPW * (warp / MT); }
    static __device__ __forceinline__ int place(int r, int d) { return r * D + (d ^ ((r & 3) << 3)); }
    static __device__ __forceinline__ int row(int warp, int lane, int e) { return 16 * (warp % MT) + (lane >> 2) + 8 * e; }
    __device__ __forceinline__ void fetch(const DecodeArgs &a, const Span &sp, int h, int warp, int lane) {
        const int rows = a.G * sp.n;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row(warp, lane, e), t = r / a.G;
            const uint16_t *const q = a.q + (static_cast<size_t>(sp.row0 + t) * a.heads + static_cast<size_t>(h) * a.G + (r - t * a.G)) * D +
                                      2 * (lane & 3);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                qf[ks][e] = r < rows ? __ldg(reinterpret_cast<const uint32_t *>(q + 16 * ks)) : 0u;
                qf[ks][2 + e] = r < rows ? __ldg(reinterpret_cast<const uint32_t *>(q + 16 * ks + 8)) : 0u;
            }
            pos[e] = sp.len - sp.n + min(t, sp.n - 1);
        }
    }
    __device__ __forceinline__ void begin() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
        lp[0] = lp[1] = lp[2] = lp[3] = 0.f;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    }
    __device__ __forceinline__ void tile(const DecodeArgs &a, uint32_t sk, uint32_t sv, int j0, bool all_seen, int warp, int lane) {
        float s[KPW / 8][4], top[2] = {-INFINITY, -INFINITY}, safe[2];
#pragma unroll
        for (int nb = 0; nb < KPW / 16; ++nb) {
            float(&s0)[4] = s[2 * nb], (&s1)[4] = s[2 * nb + 1];
            s0[0] = s0[1] = s0[2] = s0[3] = s1[0] = s1[1] = s1[2] = s1[3] = 0.f;
            // matrices: keys +0..7 / +8..15 (lane bit 4), channels +0..7 / +8..15 (lane bit 3)
            const int r = keys0(warp) + 16 * nb + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const int ch = 2 * ks + ((lane >> 3) & 1);
                uint32_t b[4];
                ldsm4(sk + r * D * 2 + ((ch ^ (r & 7)) << 4), b);
                mma16816(s0, qf[ks], b[0], b[1]);
                mma16816(s1, qf[ks], b[2], b[3]);
            }
        }
#pragma unroll
        for (int nb = 0; nb < KPW / 8; ++nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[nb][e] = seen_score(a, s[nb][e], all_seen, j0 + 8 * nb + 2 * (lane & 3) + (e & 1), pos[e >> 1]);
                top[e >> 1] = fmaxf(top[e >> 1], s[nb][e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
            const float mn = fmaxf(m[e], top[e]);
            safe[e] = mn == -INFINITY ? 0.f : mn;
            const float f = ex2(m[e] - safe[e]);
            m[e] = mn;
            l[e] *= f;
            lp[2 * e] *= f;
            lp[2 * e + 1] *= f;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
                o[d][2 * e] *= f;
                o[d][2 * e + 1] *= f;
            }
        }
#pragma unroll
        for (int nb = 0; nb < KPW / 8; ++nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[nb][e] = ex2(s[nb][e] - safe[e >> 1]);
                l[e >> 1] += s[nb][e];
            }
        }
#pragma unroll
        for (int kb = 0; kb < KPW / 16; ++kb) {
            const uint32_t p[4] = {pack_bf16(s[2 * kb][0], s[2 * kb][1]), pack_bf16(s[2 * kb][2], s[2 * kb][3]),
                                   pack_bf16(s[2 * kb + 1][0], s[2 * kb + 1][1]),
                                   pack_bf16(s[2 * kb + 1][2], s[2 * kb + 1][3])};
            mma16816(lp, p, kOnes, kOnes);
            const int r = keys0(warp) + 16 * kb + (lane & 15);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                const int ch = 2 * d + (lane >> 4);
                uint32_t b[4];
                ldsm4t(sv + r * D * 2 + ((ch ^ (r & 7)) << 4), b);
                mma16816(o[2 * d], p, b[0], b[1]);
                mma16816(o[2 * d + 1], p, b[2], b[3]);
            }
        }
    }
    __device__ __forceinline__ void put_sums(float4 *ml, int warp, int lane) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if ((lane & 3) == 0) ml[warp / MT * ROWS + row(warp, lane, e)] = make_float4(m[e], l[e], lp[2 * e], 0.f);
        }
    }
    __device__ __forceinline__ void put_o(float *so, int rows, int warp, int lane) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row(warp, lane, e);
            if (r < rows) {
                float *const w = so + (warp / MT * ROWS + r) * D + 2 * (lane & 3);
#pragma unroll
                for (int d = 0; d < D / 8; ++d)
                    *reinterpret_cast<float2 *>(w + 8 * (d ^ (r & 3))) = make_float2(o[d][2 * e], o[d][2 * e + 1]);
            }
        }
    }
};

template <int D, int R>
using Rows = std::conditional_t<R == 8, RowsShort<D>, RowsLong<D, R == 32 ? 2 : 1>>;

// D: head_dim; R: the most query rows per kv head (8, 16 or 32).
template <int D, int R>
struct DecodeCfg {
    static constexpr int kTile = tile_of(D);
    static constexpr int KG = Rows<D, R>::KG;     // key groups: warps that split a tile's keys
    static constexpr int STAGES = D == 64 ? 2 : 3;
    static constexpr int HALF = kTile * D * 2;    // bytes of a tile's K (or V)
    static constexpr int OFF_ML = STAGES * 2 * HALF;        // [KG][R] of (m, l, l of the rounded p, -)
    static constexpr int OFF_MISC = OFF_ML + KG * R * 16;   // scan, cursor, flags
    static_assert(KG * R * D * 4 <= 2 * HALF, "the warps' o go into the stage of the tile just used");
    static constexpr int BYTES = OFF_MISC + 256;
    static constexpr int CTAS = D == 64 ? 3 : 2;  // resident per SM
};

template <int D, int R>
__global__ void __launch_bounds__(kThreads, DecodeCfg<D, R>::CTAS) decode_kernel(const __grid_constant__ DecodeArgs a) {
    using C = DecodeCfg<D, R>;
    constexpr int kTile = tile_of(D);
    extern __shared__ __align__(128) uint8_t sm[];
    float4 *const sml = reinterpret_cast<float4 *>(sm + C::OFF_ML);
    long long *const sscan = reinterpret_cast<long long *>(sm + C::OFF_MISC);  // 4 warp sums
    long long *const scur = sscan + 4;                                         // sequence, its first tile
    int *const sbad = reinterpret_cast<int *>(scur + 2);                       // per stage: a needed entry is no page

    grid_release();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hk = a.c.kv_heads, part_rows = a.G * a.K;

    // ---- this CTA's run: the tiles of all sequences, summed by the whole block
    const int per = (a.N + kThreads - 1) / kThreads, n_lo = min(a.N, tid * per), n_hi = min(a.N, n_lo + per);
    long long mine = 0;
    for (int n0 = n_lo; n0 < n_hi; n0 += 4) {
        Bounds bs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) bs[k] = bounds_of(a, min(n0 + k, n_hi - 1));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            bool bad;
            const int tiles = span_of<kTile>(a, bs[k], bad).tiles;
            if (n0 + k < n_hi) {
                mine += tiles;
                if (bad && blockIdx.x == 0) atomicExch(a.status, KDA_ERR_INVALID_ARG);
            }
        }
    }
    mine *= hk;
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sscan[warp] = x;
    __syncthreads();
    long long base = x - mine, all = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < warp) base += sscan[w];
        all += sscan[w];
    }
    const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), all));
    const int cta = blockIdx.x;
    if (cta == 0 && tid == 0) a.info[0] = all;
    if (cta >= ctas) return;
    const long long t_begin = run_start(all, ctas, cta), t_end = run_start(all, ctas, cta + 1);
    if (t_begin >= base && t_begin < base + mine) {
        long long at = base;
        for (int n = n_lo; n < n_hi; ++n) {
            bool bad;
            const long long w = static_cast<long long>(span_of<kTile>(a, bounds_of(a, n), bad).tiles) * hk;
            if (t_begin < at + w) {
                scur[0] = n;
                scur[1] = at;
                break;
            }
            at += w;
        }
    }
    __syncthreads();

    // ---- cursors over (sequence, kv head, tile of the pair); both start at t_begin
    struct Cursor {
        int n, h, i;  // sequence, kv head, tile within the pair
        Span s;
        const int *table;
    };
    auto open = [&](Cursor &c) {  // the sequence's span; skips sequences without tiles
        bool bad;
        for (; c.n < a.N; ++c.n) {
            c.s = span_of<kTile>(a, bounds_of(a, c.n), bad);
            if (c.s.tiles > 0) break;
        }
        if (c.n < a.N) c.table = a.c.table + static_cast<size_t>(a.slots ? a.slots[c.n] : c.n) * a.c.max_pages;
    };
    auto step = [&](Cursor &c) {
        if (++c.i < c.s.tiles) return;
        c.i = 0;
        if (++c.h < hk) return;
        c.h = 0;
        ++c.n;
        open(c);
    };
    Cursor lc;
    lc.n = static_cast<int>(scur[0]);
    lc.h = 0;
    lc.i = 0;
    open(lc);
    {
        const long long in = t_begin - scur[1];
        lc.h = in < (1LL << 31) ? static_cast<int>(in) / lc.s.tiles : static_cast<int>(in / lc.s.tiles);
        lc.i = static_cast<int>(in - static_cast<long long>(lc.h) * lc.s.tiles);
    }
    Cursor cc = lc;
    if (tid == 0) {
        long long *const f = a.info + 1 + 5 * static_cast<long long>(cta);
        f[0] = lc.h;
        f[1] = t_begin - lc.i;
        f[2] = lc.s.tiles;
        f[3] = lc.s.row0;
        f[4] = lc.s.n;
    }

    // ---- loads. Lane l keeps the table entry of page 32 k + l of the sequence (`here`: k = chunk) and that of the next 32
    // (`next`, requested when its predecessor comes into use): read a tile ahead only, the entries' latency under load
    // stood in the way of the loads (8 x 16000 tokens, pages of 16: 102 us; 92 with pages of 64, whose entries last longer)
    const int ents = a.c.page_size >= kTile ? 1 : kTile >> a.c.page_shift;
    auto fetch = [&](int k) {
        const long long page = 32LL * k + lane;
        return (page << a.c.page_shift) < lc.s.len ? __ldg(lc.table + page) : 0;
    };
    int chunk = -1, of = -1, here = 0, next = 0;
    auto pages = [&]() {  // for the tile at lc
        if (lc.n >= a.N) return;
        const int k = tile_row0<kTile>(lc.s, lc.i) >> (a.c.page_shift + 5);
        if (lc.n == of && k == chunk) return;
        here = lc.n == of && k == chunk + 1 ? next : fetch(k);
        next = fetch(k + 1);
        chunk = k;
        of = lc.n;
    };
    long long tl = t_begin;  // tiles requested so far
    pages();
    auto load = [&](int stage) {
        if (tl < t_end) {
            const int j0 = tile_row0<kTile>(lc.s, lc.i);
            const uint32_t sk = smem_addr(sm + stage * 2 * C::HALF), sv = sk + C::HALF;
            constexpr int CH = D / 8, RP = kThreads / CH;  // 16-byte chunks per row, rows per pass
            const int ch = tid % CH;
            const int entry = __shfl_sync(0xffffffffu, here, ((j0 >> a.c.page_shift) & 31) + (lane < ents ? lane : 0));
            // a page that some visible row of the tile needs and that is none: every warp finds the same
            const int jp = j0 + lane * a.c.page_size, je = min(min(jp + a.c.page_size, j0 + kTile), lc.s.len);
            const bool wrong = __any_sync(0xffffffffu, lane < ents && jp < lc.s.len && (je > lc.s.lo || jp < a.sinks) &&
                                                           (entry < 0 || entry >= a.c.num_pages));
            if (tid == 0) sbad[stage] = wrong;
#pragma unroll
            for (int r0 = 0; r0 < kTile; r0 += RP) {
                const int r = r0 + tid / CH, j = j0 + r;
                const int pg = __shfl_sync(0xffffffffu, entry, ents == 1 ? 0 : r >> a.c.page_shift);
                // rows that no query row sees are zeros in shared memory, whatever the page holds
                const bool live = j < lc.s.len && (j >= lc.s.lo || j < a.sinks) && pg >= 0 && pg < a.c.num_pages;
                const size_t off = live ? ((static_cast<size_t>(pg) * hk + lc.h) * a.c.page_size + (j & (a.c.page_size - 1))) * D + 8 * ch
                                        : 0;
                const uint32_t so16 = static_cast<uint32_t>(r * D * 2 + ((ch ^ (r & 7)) << 4));
                cp16(sk + so16, a.c.k + off, live);
                cp16(sv + so16, a.c.v + off, live);
            }
            step(lc);
            ++tl;
            pages();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    Rows<D, R> w;
    bool seg_bad = false;
#pragma unroll 1
    for (int s = 0; s < C::STAGES - 1; ++s) load(s);
    int stage = 0;
    long long seg0 = t_begin;  // where the current pair's tiles in this run begin
    w.fetch(a, cc.s, cc.h, warp, lane);
    w.begin();
#pragma unroll 1
    for (long long t = t_begin; t < t_end; ++t) {
        asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 2) : "memory");
        __syncthreads();  // tile t has landed for every thread, and the stage before it is free
        const bool tile_bad = sbad[stage] != 0;
        load(stage == 0 ? C::STAGES - 1 : stage - 1);
        seg_bad |= tile_bad;

        const uint32_t sk = smem_addr(sm + stage * 2 * C::HALF);
        constexpr int KPW = Rows<D, R>::KPW;
        const int j0 = tile_row0<kTile>(cc.s, cc.i) + Rows<D, R>::keys0(warp);
        // the warp's keys are all visible to every row, or each weight is looked at
        const bool all_seen = j0 + KPW <= cc.s.len - cc.s.n + 1 && (!a.window || j0 > cc.s.len - 1 - a.window);
        w.tile(a, sk, sk + C::HALF, j0, all_seen, warp, lane);
        float *const so = reinterpret_cast<float *>(sm + stage * 2 * C::HALF);  // free once all warps are here
        if (++stage == C::STAGES) stage = 0;

        // ---- the pair's last tile of this run: join the warps, then write the result or this run's part
        if (cc.i + 1 == cc.s.tiles || t + 1 == t_end) {
            const long long pair0 = t - cc.i;  // the pair's first tile in the list
            const bool whole = pair0 >= t_begin && cc.i + 1 == cc.s.tiles;
            const int slot = seg0 == t_begin ? 0 : 1, rows = a.G * cc.s.n, h = cc.h, row0 = cc.s.row0;
            if (t + 1 < t_end) {
                step(cc);
                w.fetch(a, cc.s, cc.h, warp, lane);
                seg0 = t + 1;
            }
            w.put_sums(sml, warp, lane);
            __syncthreads();
            w.put_o(so, rows, warp, lane);
            __syncthreads();
            for (int i = tid; i < rows * (D / 4); i += kThreads) {
                const int r = i / (D / 4), d = 4 * (i % (D / 4));
                float top_all = -INFINITY, sum = 0.f, sum_p = 0.f;
                float4 ml[C::KG], v = make_float4(0.f, 0.f, 0.f, 0.f), u[C::KG];
#pragma unroll
                for (int g = 0; g < C::KG; ++g) {
                    ml[g] = sml[g * R + r];
                    u[g] = *reinterpret_cast<const float4 *>(so + g * R * D + Rows<D, R>::place(r, d));
                    top_all = fmaxf(top_all, ml[g].x);
                }
                const float ref = top_all == -INFINITY ? 0.f : top_all;
#pragma unroll
                for (int g = 0; g < C::KG; ++g) {  // in key order
                    const float f = ex2(ml[g].x - ref);
                    sum = fmaf(ml[g].y, f, sum);
                    sum_p = fmaf(ml[g].z, f, sum_p);
                    v.x = fmaf(u[g].x, f, v.x);
                    v.y = fmaf(u[g].y, f, v.y);
                    v.z = fmaf(u[g].z, f, v.z);
                    v.w = fmaf(u[g].w, f, v.w);
                }
                if (whole) {
                    if (!seg_bad) {
                        const int tk = r / a.G;
                        const size_t row = static_cast<size_t>(row0 + tk) * a.heads + h * a.G + (r - tk * a.G);
                        const float inv = sum == 0.f ? 0.f : 1.f / sum_p;
                        *reinterpret_cast<uint2 *>(a.out + row * D + d) =
                            make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
                        if (a.lse && d == 0) a.lse[row] = sum == 0.f ? -INFINITY : (top_all + log2f(sum)) * kLn2;
                    }
                } else {
                    const size_t pr = (static_cast<size_t>(cta) * 2 + slot) * part_rows + r;
                    *reinterpret_cast<float4 *>(a.part_o + pr * D + d) = v;
                    if (d == 0)
                        *reinterpret_cast<float4 *>(a.part_ml + 4 * pr) = make_float4(top_all, seg_bad ? -1.f : sum, sum_p, 0.f);
                }
            }
            if (seg_bad && tid == 0) atomicExch(a.status, KDA_ERR_INVALID_ARG);
            // the next tile's barrier comes before anything goes into so or sml again
            w.begin();
            seg_bad = false;
        } else {
            ++cc.i;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// The pair that the cut between runs c - 1 and c splits, if that is the pair's first cut: the parts of its rows, added
// in a fixed order. WIDE: block (c - 1, r) takes row r, every warp every fourth part (a few pairs in many
// parts); else a warp takes a row and all its parts (many pairs in two or three, and four times fewer blocks).
constexpr int kJoinWarps = 4;
template <int D, bool WIDE>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ DecodeArgs a, int grid_ctas) {
    constexpr int E = D / 32, STEP = WIDE ? kJoinWarps : 1;
    __shared__ float so[kJoinWarps][WIDE ? D : 1];
    __shared__ float3 sml[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = a.G * a.K;
    const int c = blockIdx.x + 1, r = WIDE ? blockIdx.y : kJoinWarps * blockIdx.y + warp;
    const long long *const f = a.info + 1 + 5LL * c;
    grid_acquire();
    const long long all = a.info[0], h = f[0], first = f[1], tiles = f[2], row0 = f[3], n = f[4];  // one round of reads
    const int ctas = static_cast<int>(min(static_cast<long long>(grid_ctas), all));
    if (c >= ctas || r >= a.G * n || run_start(all, ctas, c) == first) return;
    const long long before = run_start(all, ctas, c - 1);
    if (before > first) return;
    const int last = run_of(all, ctas, first + tiles - 1), slot0 = before == first ? 0 : 1;
    auto at = [&](int k) { return (static_cast<size_t>(k) * 2 + (k == c - 1 ? slot0 : 0)) * rows + r; };

    float m = -INFINITY, l = 0.f, lp = 0.f, v[E];
    bool bad = false;  // a part met a page that is none
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.f;
#pragma unroll 4
    for (int k = c - 1 + (WIDE ? warp : 0); k <= last; k += STEP) {
        const float4 ml = *reinterpret_cast<const float4 *>(a.part_ml + 4 * at(k));
        const float *const src = a.part_o + at(k) * D + E * lane;
        float x[E];
        if constexpr (E == 4) {
            const float4 q = *reinterpret_cast<const float4 *>(src);
            x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
        } else {
            const float2 q = *reinterpret_cast<const float2 *>(src);
            x[0] = q.x, x[1] = q.y;
        }
        bad |= ml.y == -1.f;
        const float mn = fmaxf(m, ml.x), ref = mn == -INFINITY ? 0.f : mn, w0 = ex2(m - ref), w1 = ex2(ml.x - ref);
        m = mn;
        l = fmaf(l, w0, ml.y * w1);
        lp = fmaf(lp, w0, ml.z * w1);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = fmaf(v[e], w0, x[e] * w1);
    }
    const int tk = r / a.G;
    const size_t row = static_cast<size_t>(row0 + tk) * a.heads + h * a.G + (r - tk * a.G);
    if constexpr (!WIDE) {
        if (bad) return;
        const float inv = l == 0.f ? 0.f : 1.f / lp;
        uint32_t u[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2) u[e / 2] = pack_bf16(v[e] * inv, v[e + 1] * inv);
        uint16_t *const dst = a.out + row * D + E * lane;
        if constexpr (E == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(u[0], u[1]);
        else *reinterpret_cast<uint32_t *>(dst) = u[0];
        if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) so[warp][E * lane + e] = v[e];
        if (lane == 0) sml[warp] = make_float3(m, l, lp);
        if (__syncthreads_or(bad)) return;
        if (threadIdx.x >= D) return;  // D <= 32 kJoinWarps
        float top = -INFINITY, o = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, sml[w].x);
        const float ref = top == -INFINITY ? 0.f : top;
        l = lp = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            const float f1 = ex2(sml[w].x - ref);
            o = fmaf(so[w][threadIdx.x], f1, o);
            l = fmaf(sml[w].y, f1, l);
            lp = fmaf(sml[w].z, f1, lp);
        }
        a.out[row * D + threadIdx.x] = f32_to_bf16(l == 0.f ? 0.f : o / lp);
        if (a.lse && threadIdx.x == 0) a.lse[row] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
    }
}

template <int D, int R>
int launch_decode(const DecodeArgs &a, int grid, cudaStream_t s) {
    using C = DecodeCfg<D, R>;
    static std::atomic<unsigned long long> attr{0};
    KDA_TRY(smem_opt_in(decode_kernel<D, R>, C::BYTES, attr, true));
    decode_kernel<D, R><<<grid, kThreads, C::BYTES, s>>>(a);
    KDA_TRY(launch_status());
    if (grid < 2) return KDA_OK;
    const int rows = a.G * a.K;
    if (static_cast<long long>(a.N) * a.c.kv_heads * 8 < grid)
        return launch_after(join_kernel<D, true>, dim3(grid - 1, rows), dim3(32 * kJoinWarps), 0, s, a, grid);
    return launch_after(join_kernel<D, false>, dim3(grid - 1, (rows + kJoinWarps - 1) / kJoinWarps), dim3(32 * kJoinWarps), 0,
                        s, a, grid);
}

int ctas_per_sm(int D) { return D == 64 ? 3 : 2; }

size_t info_bytes(int grid) { return (1 + 5 * static_cast<size_t>(grid)) * 8 / 16 * 16 + 16; }

}  // namespace

size_t attn_rows_scratch_bytes(int K, int heads, const kda_kv_cache *cache) {
    const size_t rows = static_cast<size_t>(heads / cache->kv_heads) * K;
    const int grid = ctas_per_sm(cache->head_dim) * num_sms();
    return info_bytes(grid) + static_cast<size_t>(grid) * 2 * rows * (cache->head_dim + 4) * sizeof(float);
}

int attn_rows(const kda_kv_cache *cache, int layer, const uint16_t *q, const int *cu, const int *slots, int N, int K,
              int total, int window, int sinks, uint16_t *out, float *lse, void *scratch, const kda_dims *dims,
              cudaStream_t s) {
    DecodeArgs a{};
    a.c = kv_view(cache, layer);
    a.q = q;
    a.cu = cu;
    a.slots = slots;
    a.out = out;
    a.lse = lse;
    a.status = device_status_ptr();
    if (!a.status) return KDA_ERR_CUDA;
    a.N = N;
    a.K = K;
    a.total = total;
    a.G = dims->heads / cache->kv_heads;
    a.heads = dims->heads;
    // a window that holds the longest sequence is none
    a.window = window < a.c.max_pages * a.c.page_size ? window : 0;
    a.sinks = std::min(sinks, a.c.max_pages * a.c.page_size);
    a.scale2 = dims->scale * kLog2e;
    const int rows = a.G * K, D = dims->head_dim;
    const int grid = ctas_per_sm(D) * num_sms();
    char *const p = static_cast<char *>(scratch);
    a.info = reinterpret_cast<long long *>(p);
    a.part_o = reinterpret_cast<float *>(p + info_bytes(grid));
    a.part_ml = a.part_o + static_cast<size_t>(grid) * 2 * rows * D;
    if (D == 128)
        return rows <= 8 ? launch_decode<128, 8>(a, grid, s)
                         : (rows <= 16 ? launch_decode<128, 16>(a, grid, s) : launch_decode<128, 32>(a, grid, s));
    return rows <= 8 ? launch_decode<64, 8>(a, grid, s)
                     : (rows <= 16 ? launch_decode<64, 16>(a, grid, s) : launch_decode<64, 32>(a, grid, s));
}

namespace {

int check_shape(int N, int K, const kda_dims *dims, const kda_kv_cache *cache) {
    KDA_TRY(check_cache(cache));
    KDA_TRY(check_dims(dims));
    if (N < 0 || K < 0) return KDA_ERR_INVALID_ARG;
    if (dims->head_dim != cache->head_dim || dims->heads % cache->kv_heads) return KDA_ERR_INVALID_ARG;
    if (static_cast<long long>(dims->heads / cache->kv_heads) * K > 64) return KDA_ERR_UNSUPPORTED;
    if (static_cast<long long>(N) * K > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    if (!few_rows(K, dims->heads, cache) && !attn_tiles_fits(N, N * K, dims->heads, cache)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_attn_decode_scratch_bytes(int N, int K, const kda_dims *dims, const kda_kv_cache *cache) {
    if (kda::check_shape(N, K, dims, cache) != KDA_OK || N == 0 || K == 0) return 0;
    return kda::few_rows(K, dims->heads, cache) ? kda::attn_rows_scratch_bytes(K, dims->heads, cache)
                                                : kda::attn_tiles_scratch_bytes(N, N * K, dims->heads, cache);
}

int kda_attn_decode(const kda_kv_cache *cache, int layer, const kda_bf16 *q, const int *slots, int N, int K, int window,
                    int sinks, kda_bf16 *out, float *lse, void *scratch, size_t scratch_bytes, const kda_dims *dims,
                    void *stream) {
    KDA_TRY(kda::check_shape(N, K, dims, cache));
    if (!q || !out || window < 0 || sinks < 0 || layer < 0 || layer >= cache->layers) return KDA_ERR_INVALID_ARG;
    if (!kda::aligned16(q) || !kda::aligned16(out)) return KDA_ERR_MISALIGNED;
    if (N == 0 || K == 0) return KDA_OK;
    KDA_TRY(kda::check_scratch(scratch, scratch_bytes, kda_attn_decode_scratch_bytes(N, K, dims, cache)));
    auto s = static_cast<cudaStream_t>(stream);
    if (kda::few_rows(K, dims->heads, cache))
        return kda::attn_rows(cache, layer, q, nullptr, slots, N, K, N * K, window, sinks, out, lse, scratch, dims, s);
    return kda::attn_tiles(cache, layer, q, nullptr, slots, N, K, N * K, window, sinks, out, lse, scratch, dims, s);
}

}  // extern "C"
