// Attention of packed query rows over their paged cache (include/kda.h, kda_attn_prefill).
//
// Per (sequence, kv head) the n query tokens of G query heads are n G rows (token major, then head), cut into tiles of
// 256 (128 at head_dim 64); a CTA takes one such tile and walks the visible rows of the cache once, 128 at a time, with
// the softmax's running reference m and sum l: S = Q K^T, P = 2^(scale log2(e) S - m), l += rowsum P, O += P V.
// 4 D flops and one exponential per (row, cached row) pair: the tensor cores bound it at D = 128 (512 cycles of MMA for each
// 128 x 128 x 128 product; 256 rows by 128 keys are four of them and 2048 cycles of exponentials), the exponentials at D = 64.
//
// Warps (the softmax warps take registers that the last four give up, as setmaxnreg's comment there says):
//   softmax     four per 128 rows, one row per thread, so that no shuffles are needed: S from TMEM, mask at the edges, P as
//               BF16 back into TMEM; also Q into shared memory at the start and O out at the end
//   TMA         K and V page by page (one box of 64 channels per page, at most 128 rows), 128-byte swizzle, two stages; V of a
//               tile and K of the next share a barrier
//   MMA         tcgen05.mma, P as the A operand from TMEM, taken in two halves of 64 keys as the softmax finishes them. At
//               D = 128 two halves of rows alternate: P_a V, next S_a, P_b V, next S_b, so that one half's products run under
//               the other's softmax, and P lies over its S (TMEM columns: S_a 0, S_b 128, O_a 256, O_b 384). At D = 64 a
//               CTA has one half and two CTAs share an SM; P has columns of its own (S 0, O 128, P 192), so that the
//               next S is formed as soon as this one is in registers.
//   zeros       in the V rows of edge tiles that no row of the CTA sees
// O is rescaled only when a row's maximum has grown by more than 2^8 since its reference was set (P then
// stays below 2^8, harmless in BF16 and FP32). P is rounded to BF16 for the second product (at most 2^-8 of each weight).
// O is divided by the sum of the rounded weights, as in the one-token form, so that a row that few keys carry is not scaled by
// their roundings (V rows that are all alike come out as they are); lse takes the sum of the unrounded ones. The second
// sum costs two additions per pair of weights: 452 us against 442 for 8192 tokens at head_dim 128, 421 against 390 at 64 (these
// are additions of BF16 to FP32; by shifts and masks 472 and 447, as products with ones by mma.sync 636 and 482).
// Where the tiles are fewer than the SMs, several CTAs share a walk and prefill_join_kernel adds their parts in order.
//
// Rows of a cache tile that no row of the CTA sees (past the last token, before the window, pages that
// left the table) are not loaded where they fill a page, and their V rows are zeroed in shared memory: what
// they hold cannot reach a result. Every wait on a barrier is bounded; one that gives up latches KDA_ERR_TIMEOUT. Only tcgen05.alloc
// waits as long as other CTAs of the SM hold its columns; each takes its columns once, so none waits for a second lot.
//
// Measured (BF16 1679 TFLOP/s in a burst, 1422 sustained): one prompt of 8192 tokens, 32 heads on 8 kv heads of 128, causal: 452 us =
// 1217 TFLOP/s in bursts of 20, 532 to 540 us = 1020 to 1034 in a loop, once the power limit holds the clocks down; 4096 tokens 132 us,
// 2048 46; head_dim 64: 421 us, 440 in a loop. A chunk of 1024 rows behind 60000 tokens: 848 us (1197 TFLOP/s), at 64 835.
// Without the second sum of weights a tile took about 2950 cycles for 256 rows at D = 128 (a row half's chain: softmax 1840, its two
// products 1220) and 3180 at D = 64. There the exponential unit was 60 % busy and the issue slots 43 %: neither is full, two softmax
// warps per scheduler do not cover each other's latencies. Before its first tile a CTA spends 6500 cycles
// (bounds, slot, length and page entry, which depend on one another; Q; K) and after its last product 3000 on O; nothing runs
// under these at D = 128. Tried and slower: the row's keys
// split between two threads (549 us: the maxima's exchange), a quarter to a half of the exponentials as polynomials on
// the FMA pipe (no gain at 128, 398 to 474 us against 386 at 64: the added instructions cost more than the unit's time saved), S read twice from TMEM instead of kept in
// registers (506), both halves' key halves with an O of their own at D = 64 (424), Q requested before the set-up's barrier (463: spills;
// later, with Q by whole rows and K of tile 0 too, 451 against 447), CTAs that take further tiles in place by cluster launch
// control, the next tile's K and Q loaded under this one's end (438 against 434, 397 against 388 at 64: what it saves between tiles,
// 3 to 5 %, the products' loop loses to stages that no longer are constants), 200 + 104 registers for 208 + 88 (449 against 446).
#include <algorithm>
#include <cmath>

#include "kv.cuh"
#include "tma.cuh"
#include "umma.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kKeys = 128;
constexpr int kSplitTiles = 4;  // the least tiles of a walk's part
constexpr long long kPrefillWait = 4000000000LL;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.0f;  // log2 of how far a maximum may outgrow its reference

struct PrefillArgs {
    CUtensorMap tk, tv;
    KvView c;
    const uint16_t *q;
    const int *cu, *slots;
    uint16_t *out;
    float *lse;
    int *status;
    int B, max_rows, total, heads, G, window, sinks, nslots;
    int splits;             // CTAs that share a tile's walk; above 1 each leaves a part
    float *part_o;          // [slot][kv head][split][256][D]
    float *part_ml;         // [slot][kv head][split][256][4]: m, l (-1: bad page), l of the rounded P
    float scale2;  // |scale| log2(e)
    uint32_t flip;  // sign bits of a BF16 pair if scale < 0 (the queries are negated), else 0
};

// Rows of a CTA's tile: see the head of the file.
__host__ __device__ constexpr int halves_of(int D) { return D == 64 ? 1 : 2; }
__host__ __device__ constexpr int tile_rows(int D) { return 128 * halves_of(D); }

template <int D>
struct PrefillCfg {
    static constexpr int NH = halves_of(D), ROWS = tile_rows(D), THREADS = 128 * (NH + 1), CTAS = NH == 1 ? 2 : 1;
    // Whether P has TMEM columns of its own: the next S can then be formed as soon as S is in registers
    static constexpr bool OWN_P = D == 64;
    // TMEM columns: S of the halves, O of the halves, P (at head_dim 128 P lies over its S)
    static constexpr int TMEM = 256 * NH, COL_O = 128 * NH, COL_P = OWN_P ? COL_O + D * NH : 0;
    static constexpr int STEP_P = OWN_P ? 64 : 128;
    static constexpr int TILE = kKeys * D * 2;  // bytes of a Q half, K or V tile
    static constexpr int OFF_K = NH * TILE, OFF_V = OFF_K + 2 * TILE, OFF_BARS = OFF_V + 2 * TILE;
    static constexpr int BYTES = OFF_BARS + 256 + 1024;
};

__device__ __forceinline__ void tma_load_2d(void *smem_dst, const CUtensorMap *tm, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// D[tmem] (+)= A[tmem] . B[smem]: A's rows are TMEM lanes, two BF16 values of K per column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// One try with the hardware's own suspend time: the waits here are short and on the critical chain (2 % faster than
// the long hint of mbar_try_wait, 8192 rows x 32 heads).
__device__ __forceinline__ uint32_t try_wait(uint32_t addr, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    return done;
}
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort, int *status) {
    const uint32_t addr = smem_u32(bar);
    if (try_wait(addr, parity)) return true;
    const long long t0 = clock64();
    while (!try_wait(addr, parity)) {
        if (*abort) return false;
        if (clock64() - t0 > kPrefillWait) {
            *abort = 1;
            atomicExch(status, KDA_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two FP32 values in one 64-bit register: the paired multiply-add and add issue once for both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// lo and hi plus the two BF16 values of u.
__device__ __forceinline__ void add_halves(float &lo, float &hi, uint32_t u) {
    asm("{\n\t.reg .b16 x, y;\n\t"
        "mov.b32 {x, y}, %2;\n\t"
        "add.rn.f32.bf16 %0, x, %0;\n\t"
        "add.rn.f32.bf16 %1, y, %1;\n\t}\n"
        : "+f"(lo), "+f"(hi)
        : "r"(u));
}

// True in one lane of a converged warp. The MMA role runs with its whole warp and branches on this around the
// instructions that one thread issues: their operands then stay warp-uniform.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r));
    return r != 0;
}

// The n lowest bits (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t ones_below(int n) { return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u); }

// Where a CTA's rows stand: the sequence's length and rows, and per half the positions and cache tiles.
struct Tile {
    int b, slot, c0, n, len, r0;  // r0: first of the 256 rows (token * G + head)
    int lo, hi;                   // visible cached rows: [lo, hi) and those below `sinks`
    int sink, start;              // leading tiles that only sinks need; the row where the others start (a box's first)
    int all, first;               // tiles of the whole walk; the first of this CTA's part
    // of this part's tiles i: those below sinks_to start at row 128 (i + first), the others at start + 128 (i + skip);
    // rows that no row of the CTA sees are in tiles up to dead_to and from dead_from on
    int sinks_to, skip, dead_to, dead_from;
    int tiles_a, tiles_b;         // of this part, per half
    int rows, base, p_hi_a, p_hi_b;  // rows in the tile, position of the sequence's first query, last positions
};
__device__ __forceinline__ int tile_row0(const Tile &t, int i) {
    return i < t.sinks_to ? (i + t.first) * kKeys : (i + t.skip) * kKeys + t.start;
}

// Whether cache tile i may have rows that no row of the CTA sees: the last tile, and where a window has
// passed the start, the sinks' tiles and those up to the window.
__device__ __forceinline__ bool has_dead_rows(const Tile &t, int i) {
    return i >= t.dead_from || i <= t.dead_to;
}

// Bounds of sequence b's rows, its slot and its length; false if one of them is none.
__device__ __forceinline__ int row_bound(const PrefillArgs &a, int b) { return a.cu ? a.cu[b] : b * a.max_rows; }
__device__ __forceinline__ bool sequence(const PrefillArgs &a, int b, int &c0, int &c1, int &slot, int &len) {
    c0 = row_bound(a, b);
    c1 = row_bound(a, b + 1);
    slot = a.slots ? a.slots[b] : b;
    len = slot >= 0 && slot < a.c.max_seqs ? a.c.len[slot] : -1;
    return c0 >= 0 && c1 >= c0 && c1 <= a.total && c1 - c0 <= a.max_rows && len >= 0 && len <= a.c.max_pages * a.c.page_size;
}

// Finds the row tile of `slot` (whole warps call): tiles of sequence b start at slot floor(c G / ROWS) + min(b, c), c its
// first row. The next sequence with rows has a larger b and a larger c, so that its slot is at least one past what the floors
// differ by, which keeps the tiles apart whatever the lengths; sequences without rows take no slots once there are
// more of them than rows before them. Every lane looks at a sequence, so one round of reads does for 32 of them;
// beyond that each round narrows the range 32 times first. False: no such tile, or its sequence is refused.
template <int ROWS>
__device__ __forceinline__ bool locate(const PrefillArgs &a, int slot, Tile &t) {
    auto first_slot = [&](int b, int c) { return static_cast<long long>(c) * a.G / ROWS + min(b, c); };
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = a.B;
    while (hi - lo > 32) {
        const int step = (hi - lo + 31) / 32, b = lo + lane * step;
        const uint32_t at_or_before = __ballot_sync(0xffffffffu, b < hi && first_slot(b, row_bound(a, b)) <= slot);
        if (!at_or_before) return false;
        lo += (31 - __clz(at_or_before)) * step;
        hi = min(hi, lo + step);
    }
    int c0 = 0, c1 = 0, s = 0, len = 0;
    bool ok = false, here = false;
    if (lo + lane < hi) {
        ok = sequence(a, lo + lane, c0, c1, s, len);
        here = first_slot(lo + lane, c0) <= slot && slot < first_slot(lo + lane + 1, c1);
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, here);
    if (!hit) return false;
    const int src = __ffs(hit) - 1;
    if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, src)) return false;
    t.b = lo + src;
    t.c0 = __shfl_sync(0xffffffffu, c0, src);
    t.n = __shfl_sync(0xffffffffu, c1, src) - t.c0;
    t.slot = __shfl_sync(0xffffffffu, s, src);
    t.len = __shfl_sync(0xffffffffu, len, src);
    const long long r0 = (slot - first_slot(t.b, t.c0)) * ROWS, all_rows = static_cast<long long>(t.n) * a.G;
    if (r0 < 0 || r0 >= all_rows) return false;
    t.r0 = static_cast<int>(r0);
    t.rows = static_cast<int>(min(static_cast<long long>(ROWS), all_rows - r0));
    t.base = t.len - t.n;
    const int p_lo = t.base + t.r0 / a.G;
    t.p_hi_a = t.base + (t.r0 + min(t.rows, 128) - 1) / a.G;
    t.p_hi_b = t.base + (t.r0 + t.rows - 1) / a.G;
    t.lo = a.window ? static_cast<int>(max(0LL, static_cast<long long>(p_lo) - a.window + 1)) : 0;
    t.hi = t.p_hi_b + 1;
    t.start = t.lo & ~(min(a.c.page_size, kKeys) - 1);
    t.sink = (min(a.sinks, t.lo) + kKeys - 1) / kKeys;
    if (t.sink * kKeys >= t.start) t.sink = t.start = 0;  // one walk from the first row
    t.tiles_a = t.p_hi_a < 0 ? 0 : t.sink + (t.p_hi_a - t.start) / kKeys + 1;
    t.tiles_b = t.rows <= 128 || t.p_hi_b < 0 ? 0 : t.sink + (t.p_hi_b - t.start) / kKeys + 1;
    t.all = max(t.tiles_a, t.tiles_b);
    t.first = 0;
    return true;
}

// Into how many parts a tile's walk is cut: short walks are not.
__device__ __forceinline__ int parts_of(const PrefillArgs &a, const Tile &t) {
    return min(a.splits, max(1, t.all / kSplitTiles));
}

template <int D>
__global__ void __launch_bounds__(PrefillCfg<D>::THREADS, PrefillCfg<D>::CTAS) prefill_kernel(const __grid_constant__ PrefillArgs a) {
    using C = PrefillCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // full[s]: V of tile i and K of tile i + 1, i % 2 = s, have landed ; empty[s]: they are read; first_k and
    // first_read: the same for K of tile 0
    uint64_t *const full = reinterpret_cast<uint64_t *>(sm + C::OFF_BARS);
    uint64_t *const empty = full + 2, *const first_k = empty + 2, *const first_read = first_k + 1;
    uint64_t *const sfull = first_read + 1, *const pfull = sfull + 2, *const ofull = pfull + 4, *const vfix = ofull + 2;
    uint64_t *const fixgo = vfix + 2, *const qfull = fixgo + 2, *const sfree = qfull + 1;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(sfree + 2);
    volatile int *const abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *const bad_page = abort + 1;

    constexpr int W = 4 * C::NH;  // the softmax warps come first
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int hk = a.c.kv_heads, split = blockIdx.x % a.splits, h = blockIdx.x / a.splits % hk;
    const int slot_id = a.nslots - 1 - static_cast<int>(blockIdx.x / a.splits / hk);  // the longest walks first

    // TMEM and barriers by two of the warps that do not compute, under every warp's search for the tile
    if (warp == W + 3) {  // CTA b looks sequence b over, and where there are fewer CTAs its other lanes those further on
        const long long b = blockIdx.x + static_cast<long long>(lane) * gridDim.x;  // the grid is at least B / 32
        int c0, c1, s, len;
        if (b < a.B && !sequence(a, static_cast<int>(b), c0, c1, s, len)) atomicExch(a.status, KDA_ERR_INVALID_ARG);
    }
    if (warp == W + 2 && lane == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&sfull[s], 1);
            mbar_init(&pfull[s], 4);
            mbar_init(&pfull[2 + s], 4);
            mbar_init(&vfix[s], 1);
            mbar_init(&fixgo[s], 1);
            mbar_init(&sfree[s], 4);
            mbar_init(&ofull[s], 1);
        }
        mbar_init(qfull, W);
        mbar_init(first_k, 1);
        mbar_init(first_read, 1);
        *abort = 0;
        *bad_page = 0;
        fence_mbar_init();
    }
    if (warp == W + 1) {
        tmem_alloc(tmem_slot, C::TMEM);
        tmem_relinquish();
    }

    Tile t;
    const bool found = locate<C::ROWS>(a, slot_id, t);
    const int splits = found ? parts_of(a, t) : 0;
    if (split >= splits) {  // nothing to do here but to give the columns back
        __syncthreads();
        if (warp == W + 1) tmem_dealloc(*tmem_slot, C::TMEM);
        return;
    }
    t.first = static_cast<int>(static_cast<long long>(t.all) * split / splits);
    const int ntiles = static_cast<int>(static_cast<long long>(t.all) * (split + 1) / splits) - t.first;
    t.sinks_to = t.sink - t.first;
    t.skip = t.first - t.sink;
    t.dead_to = t.lo > 0 ? t.sinks_to + (t.lo - t.start + kKeys - 1) / kKeys - 1 : -1;
    t.dead_from = t.all - 1 - t.first;
    t.tiles_a = min(max(t.tiles_a - t.first, 0), ntiles);
    t.tiles_b = min(max(t.tiles_b - t.first, 0), ntiles);

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_release();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    if (warp >= W) {
      // 384 x 168 = 256 x 208 + 128 x 88 registers, or 256 x 128 = 128 x 200 + 128 x 56
      if constexpr (C::NH == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
      else asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      if (warp == W) {
        // ---- TMA: lane l brings box l of a tile (page l / (D / 64), 64-channel half l % (D / 64))
        constexpr int HALVES = D / 64;
        const int box_rows = min(a.c.page_size, kKeys), boxes = kKeys / box_rows * HALVES;
        const int sub = lane / HALVES, half = lane % HALVES;
        const int *const table = a.c.table + static_cast<size_t>(t.slot) * a.c.max_pages;
        auto entry_of = [&](int i, bool &need) {
            const int j = tile_row0(t, i) + sub * box_rows, je = min(j + box_rows, t.hi);
            need = i < ntiles && lane < boxes && j < t.hi && (je > t.lo || j < a.sinks);
            return need ? __ldg(table + (j >> a.c.page_shift)) : 0;
        };
        struct Box {
            bool use;
            int y;
        };
        // this lane's box of tile i, and what it adds to the barrier's bytes (all lanes call)
        auto box_of = [&](int i, int entry, bool need) {
            const int j = tile_row0(t, i) + sub * box_rows;
            const bool page = entry >= 0 && entry < a.c.num_pages;
            if (need && !page) *bad_page = 1;
            return Box{need && page, page ? (entry * hk + h) * a.c.page_size + (j & (a.c.page_size - 1)) : 0};
        };
        auto bytes_of = [&](const Box &b) { return __popc(__ballot_sync(0xffffffffu, b.use)) * box_rows * 128u; };
        const uint32_t off = half * (kKeys * 128) + sub * box_rows * 128;
        bool need = false;
        int entry = entry_of(0, need), issued = 0;
        Box now = box_of(0, entry, need);
        if (ntiles > 0) {
            const uint32_t bytes = bytes_of(now);
            if (lane == 0) mbar_expect_tx(first_k, bytes);
            __syncwarp();
            if (now.use) tma_load_2d(sm + C::OFF_K + off, &a.tk, 64 * half, now.y, first_k);
        }
        entry = entry_of(1, need);
        for (int i = 0; i < ntiles; ++i) {
            const int s = i & 1;
            const Box next = box_of(i + 1, entry, need);
            const uint32_t bytes = bytes_of(now) + bytes_of(next);
            entry = entry_of(i + 2, need);  // in flight while this tile's stage comes free
            if (!wait_or_abort(&empty[s], ((i >> 1) & 1) ^ 1, abort, a.status)) break;
            if (i == 1 && !wait_or_abort(first_read, 0, abort, a.status)) break;  // K of tile 2 goes where K of tile 0 was
            if (lane == 0) mbar_expect_tx(&full[s], bytes);
            __syncwarp();
            if (now.use) tma_load_2d(sm + C::OFF_V + s * C::TILE + off, &a.tv, 64 * half, now.y, &full[s]);
            if (next.use) tma_load_2d(sm + C::OFF_K + (s ^ 1) * C::TILE + off, &a.tk, 64 * half, next.y, &full[s]);
            if (lane == 0 && has_dead_rows(t, i)) mbar_arrive(&fixgo[s]);
            issued = i + 1;
            now = next;
        }
        if (*abort && ntiles > 0) {  // nobody consumes what is in flight any more: let it land before the CTA ends
            mbar_wait(first_k, 0, 100000000LL);
            for (int i = max(0, issued - 2); i < issued; ++i) mbar_wait(&full[i & 1], (i >> 1) & 1, 100000000LL);
        }
      } else if (warp == W + 1) {
        // ---- MMA; what it waits for is nearly always there but P
        if (ntiles > 0) {
            constexpr uint32_t id_s = idesc_bf16(128, kKeys, false, false), id_o = idesc_bf16(128, D, false, true);
            const uint32_t sq = smem_u32(sm);
            uint32_t fixes = 0;  // bit s: parity of the next zeroed V tile in stage s
            auto commit = [&](uint64_t *bar) {
                if (elect_one()) mma_commit(bar);
                __syncwarp();
            };
            auto scores = [&](int x, int i) {  // S_x = Q_x K_i^T
                const uint64_t dq = kmaj_desc(sq + x * C::TILE, 128, 0, 0);
                const uint64_t dk = kmaj_desc(sq + C::OFF_K + (i & 1) * C::TILE, kKeys, 0, 0);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_bf16(tmem + 128 * x, dq + kmaj_step(128, ks), dk + kmaj_step(kKeys, ks), id_s, ks > 0);
                    mma_commit(&sfull[x]);
                }
                __syncwarp();
            };
            // tile i's V and tile i + 1's K
            auto operands = [&](int i) {
                const int s = i & 1;
                bool ok = wait_or_abort(&full[s], (i >> 1) & 1, abort, a.status);
                if (ok && has_dead_rows(t, i)) {
                    ok = wait_or_abort(&vfix[s], (fixes >> s) & 1, abort, a.status);
                    fixes ^= 1u << s;
                }
                return ok;
            };
            bool ok = wait_or_abort(qfull, 0, abort, a.status) && wait_or_abort(first_k, 0, abort, a.status);
            if (ok) {
                tc_fence_after();
                if (t.tiles_a > 0) scores(0, 0);
                if (C::NH == 2 && t.tiles_b > 0) scores(1, 0);
                commit(first_read);
                ok = operands(0);
            }
            for (int i = 0; ok && i < ntiles; ++i) {
                const int s = i & 1;
                const uint64_t dv = mnmaj_desc(sq + C::OFF_V + s * C::TILE, kKeys, 0, 0);
#pragma unroll
                for (int x = 0; x < C::NH; ++x) {
                    const int tiles = x ? t.tiles_b : t.tiles_a;
                    if (ok && i < tiles) {
                        if (C::OWN_P && i + 1 < tiles) {
                            if (!(ok = wait_or_abort(&sfree[x], i & 1, abort, a.status))) break;
                            tc_fence_after();
                            scores(x, i + 1);
                        }
#pragma unroll
                        for (int half = 0; half < 2; ++half) {  // P comes in two halves of 64 keys
                            if (ok) ok = wait_or_abort(&pfull[2 * half + x], i & 1, abort, a.status);
                            if (!ok) break;
                            tc_fence_after();
                            if (elect_one()) {
#pragma unroll
                                for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
                                    mma_bf16_ta(tmem + C::COL_O + D * x, tmem + C::COL_P + C::STEP_P * x + 8 * ks, dv + mnmaj_step(ks), id_o, i > 0 || ks > 0);
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                        if (C::OWN_P || i + 1 == tiles) commit(&ofull[x]);
                        else scores(x, i + 1);
                    }
                }
                if (ok && i + 1 < ntiles) {  // the next operands are looked for while S_b is still running
                    commit(&empty[s]);
                    ok = operands(i + 1);
                }
            }
        }
      } else if (warp == W + 2) {
        // ---- V rows that no row of this CTA sees: zeros. fixgo says that the tile's load is under way, so that
        // full's phase is the tile's own (tiles without such rows pass unseen here)
        uint32_t gone = 0;
        for (int i = 0; i < ntiles; ++i) {
            if (!has_dead_rows(t, i)) continue;
            uint8_t *const sv = sm + C::OFF_V + (i & 1) * C::TILE;
            if (!wait_or_abort(&fixgo[i & 1], (gone >> (i & 1)) & 1, abort, a.status)) break;
            gone ^= 1u << (i & 1);
            if (!wait_or_abort(&full[i & 1], (i >> 1) & 1, abort, a.status)) break;
            const int j0 = tile_row0(t, i);
            // a row is 128 bytes of each 64-channel half, in whatever order the swizzle keeps them
            const int hi = t.hi - j0, lo = t.lo - j0, sinks = a.sinks - j0;
            for (int e = lane; e < kKeys * (D / 8); e += 32) {
                const int r = e / 8 % kKeys;
                if (r >= hi || (r < lo && r >= sinks)) *reinterpret_cast<uint4 *>(sv + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&vfix[i & 1]);
        }
      }
    } else {
        if constexpr (C::NH == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---- softmax: this thread's row of half x
        const int x = warp >> 2, r = 128 * x + 32 * (warp & 3) + lane;
        const bool real = r < t.rows;
        const int tok = (t.r0 + r) / a.G, g = t.r0 + r - tok * a.G;
        const size_t row = static_cast<size_t>(t.c0 + (real ? tok : 0)) * a.heads + static_cast<size_t>(h) * a.G + (real ? g : 0);
        const int pos = t.base + min(tok, t.n - 1);
        constexpr int LR = D / 8, RP = 32 / LR;  // lanes per row and rows per pass of Q's and O's copies
        {
            uint8_t *const rows_sm = sm + x * C::TILE + 32 * (warp & 3) * 128;
            const uint32_t reals = __ballot_sync(0xffffffffu, real);
            // D / 8 lanes bring a row: 3100 cycles at head_dim 128; where every lane brought its own, 5700
#pragma unroll
            for (int k = 0; k < LR; ++k) {
                const int of = RP * k + lane / LR;
                const size_t from = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(row), of);
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (reals >> of & 1u) v = __ldg(reinterpret_cast<const uint4 *>(a.q + from * D) + lane % LR);
                v.x ^= a.flip;
                v.y ^= a.flip;
                v.z ^= a.flip;
                v.w ^= a.flip;
                *reinterpret_cast<uint4 *>(rows_sm + kmaj_off(of, 8 * (lane % LR), 128)) = v;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull);
        }
        const uint32_t ts = tmem_lane_base(tmem, warp) + 128 * x, to = tmem_lane_base(tmem, warp) + C::COL_O + D * x;
        const uint32_t tp = tmem_lane_base(tmem, warp) + C::COL_P + C::STEP_P * x;
        const int p_first = t.base + (t.r0 + 128 * x) / a.G, p_last = x ? t.p_hi_b : t.p_hi_a, tiles = x ? t.tiles_b : t.tiles_a;
        float m = -INFINITY, l = 0.f, lr = 0.f;  // lr: the sum of the rounded weights
        bool ok = true;
        for (int i = 0; i < tiles; ++i) {
            if (!(ok = wait_or_abort(&sfull[x], i & 1, abort, a.status))) break;
            tc_fence_after();
            float s[kKeys];
#pragma unroll
            for (int c = 0; c < kKeys; c += 32) tmem_ld32(ts + c, s + c);
            tmem_ld_wait();
            if (C::OWN_P) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfree[x]);
            }
            const int j0 = tile_row0(t, i);
            if (j0 + kKeys - 1 > p_first || (a.window && j0 <= p_last - a.window)) {
                // one bit per column: [first, pos] and the sinks, as shifts of ones
                const int last = pos - j0, first = a.window ? last - a.window + 1 : -j0, sink = a.sinks - j0;
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) {
                    const uint32_t to_pos = ones_below(last + 1 - c);
                    const uint32_t seen = to_pos & (~ones_below(first - c) | ones_below(sink - c));
#pragma unroll
                    for (int e = 0; e < 32; ++e) s[c + e] = seen & (1u << e) ? s[c + e] : -INFINITY;
                }
            }
            float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < kKeys - 4; c += 8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) top[e] = max3(top[e], s[c + e], s[c + 4 + e]);
            }
            const float mn = max3(max3(top[0], s[kKeys - 4], s[kKeys - 3]), max3(top[1], s[kKeys - 2], s[kKeys - 1]),
                                  fmaxf(top[2], top[3])) * a.scale2;
            if (C::OWN_P && i > 0) {  // O and the columns of P are the last product's until it is done
                if (!(ok = wait_or_abort(&ofull[x], (i - 1) & 1, abort, a.status))) break;
                tc_fence_after();
            }
            float f = 1.f;
            if (mn > m + kGrow || m == -INFINITY) {  // -inf: the first rows this one sees; its O is still zero
                const float mx = fmaxf(m, mn);
                f = m == -INFINITY ? 0.f : ex2(m - mx);
                m = mx;
            }
            if (i > 0 && __any_sync(0xffffffffu, f != 1.f && l != 0.f)) {
#pragma unroll
                for (int c = 0; c < D; c += 16) {
                    float o[16];
                    tmem_ld16(to + c, o);
                    tmem_ld_wait();
                    uint32_t u[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * f);
                    tmem_st16(to + c, u);
                }
            }
            l *= f;
            lr *= f;
            const float ref = m == -INFINITY ? 0.f : m;
            const uint64_t scale_2 = pair(a.scale2, a.scale2), ref_2 = pair(-ref, -ref);
            uint64_t sum[2] = {0ull, 0ull};
            float rsum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kKeys; c += 32) {
                uint32_t u[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float p0, p1;
                    unpair(fma2(pair(s[c + 2 * e], s[c + 2 * e + 1]), scale_2, ref_2), p0, p1);
                    p0 = ex2(p0);
                    p1 = ex2(p1);
                    sum[e & 1] = add2(sum[e & 1], pair(p0, p1));
                    u[e] = pack_bf16(p0, p1);
                }
                tmem_st16(tp + c / 2, u);
#pragma unroll
                for (int e = 0; e < 16; ++e) add_halves(rsum[e & 1], rsum[2 + (e & 1)], u[e]);
                if (c == 32 || c == 96) {  // 64 keys' weights are there: their half of the product may start
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pfull[(c == 96 ? 2 : 0) + x]);
                }
            }
            float sum_lo, sum_hi;
            unpair(add2(sum[0], sum[1]), sum_lo, sum_hi);
            l += sum_lo + sum_hi;
            lr += (rsum[0] + rsum[1]) + (rsum[2] + rsum[3]);
        }
        // a half that sees nothing waits for the other, so that both know of a bad page
        if (ok && tiles > 0) ok = wait_or_abort(&ofull[x], C::OWN_P ? (tiles - 1) & 1 : 0, abort, a.status);
        else if (ok && ntiles > 0) ok = wait_or_abort(&ofull[x ^ 1], 0, abort, a.status);
        tc_fence_after();
        if (splits > 1) {  // this part's sums, m and unscaled O; l = -1: a page was none
            const size_t pr = (static_cast<size_t>(slot_id) * hk + h) * a.splits * C::ROWS + static_cast<size_t>(split) * C::ROWS + r;
            float4 *const dst = reinterpret_cast<float4 *>(a.part_o + pr * D);
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                float o[16];
                tmem_ld16(to + c, o);
                tmem_ld_wait();
                if (real && l != 0.f) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) dst[(c + e) / 4] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
            *reinterpret_cast<float4 *>(a.part_ml + 4 * pr) = make_float4(m, ok && !*bad_page ? l : -1.f, lr, 0.f);
            if (*bad_page && tid == 0) atomicExch(a.status, KDA_ERR_INVALID_ARG);
        } else if (__all_sync(0xffffffffu, ok && !*bad_page)) {
            const float inv = l == 0.f ? 0.f : 1.f / lr;
            uint8_t *const rows_sm = sm + x * C::TILE + 32 * (warp & 3) * 128;  // Q has been read
            int ln = lane;  // hidden from the compiler, which would keep the addresses of Q's copy in registers for this one
            asm volatile("" : "+r"(ln));
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(to + c, o);
                tmem_ld_wait();
                if (tiles == 0 || l == 0.f) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    const uint4 u = make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                                               pack_bf16(o[e + 4] * inv, o[e + 5] * inv), pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
                    if (D == 128) *reinterpret_cast<uint4 *>(rows_sm + kmaj_off(ln, c + e, 128)) = u;
                    else if (real) *reinterpret_cast<uint4 *>(a.out + row * D + c + e) = u;
                }
            }
            // whole rows at a time through shared memory (8192 rows x 32 heads: 452 us with Q and O by own rows, 441 so); at
            // head_dim 64 a row is one 128-byte line, and a lane writes its own (387 us against 389)
            if (D == 128) {
                const uint32_t reals = __ballot_sync(0xffffffffu, real);
                __syncwarp();
                uint4 v[LR];
#pragma unroll
                for (int k = 0; k < LR; ++k)
                    v[k] = *reinterpret_cast<const uint4 *>(rows_sm + kmaj_off(RP * k + ln / LR, 8 * (ln % LR), 128));
#pragma unroll
                for (int k = 0; k < LR; ++k) {
                    const size_t at = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(row), RP * k + ln / LR);
                    if (reals >> (RP * k + ln / LR) & 1u) *(reinterpret_cast<uint4 *>(a.out + at * D) + ln % LR) = v[k];
                }
            }
            if (a.lse && real) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        } else if (*bad_page && tid == 0) {
            atomicExch(a.status, KDA_ERR_INVALID_ARG);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W + 1) tmem_dealloc(tmem, C::TMEM);
}

// The parts of split walks, added in order; one warp per row.
template <int D>
__global__ void __launch_bounds__(256) prefill_join_kernel(const __grid_constant__ PrefillArgs a) {
    constexpr int E = D / 32, R = tile_rows(D);
    grid_acquire();
    const int hk = a.c.kv_heads, h = blockIdx.x % hk, slot = blockIdx.x / hk, lane = threadIdx.x & 31;
    Tile t;
    if (!locate<R>(a, slot, t)) return;
    const int splits = parts_of(a, t);
    if (splits == 1) return;
    const float4 *const ml = reinterpret_cast<const float4 *>(a.part_ml) + (static_cast<size_t>(slot) * hk + h) * a.splits * R;
    const float *const po = a.part_o + (static_cast<size_t>(slot) * hk + h) * a.splits * R * D;
    const int r = 8 * blockIdx.y + (threadIdx.x >> 5);
    if (r >= t.rows) return;
    float m = -INFINITY;
    bool bad = false;
    for (int p = 0; p < splits; ++p) {
        m = fmaxf(m, ml[p * R + r].x);
        bad |= ml[p * R + r].y == -1.f;
    }
    // a page that is none leaves the whole tile, as an unsplit walk does
    for (int p = 0; p < splits; ++p)
        for (int k = lane; k < t.rows; k += 32) bad |= ml[p * R + k].y == -1.f;
    if (__any_sync(0xffffffffu, bad)) return;
    float l = 0.f, lr = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int p = 0; p < splits; ++p) {
        const float4 part = ml[p * R + r];
        if (part.y == 0.f) continue;  // that part saw nothing and left no O
        const float w = ex2(part.x - m);
        l = fmaf(part.y, w, l);
        lr = fmaf(part.z, w, lr);
        const float *const src = po + (static_cast<size_t>(p) * R + r) * D + E * lane;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(src[e], w, o[e]);
    }
    const int q = t.r0 + r, tok = q / a.G;
    const size_t row = static_cast<size_t>(t.c0 + tok) * a.heads + static_cast<size_t>(h) * a.G + (q - tok * a.G);
    const float inv = l == 0.f ? 0.f : 1.f / lr;
    uint32_t u[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) u[e / 2] = pack_bf16(o[e] * inv, o[e + 1] * inv);
    uint16_t *const dst = a.out + row * D + E * lane;
    if constexpr (E == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(u[0], u[1]);
    else *reinterpret_cast<uint32_t *>(dst) = u[0];
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// CTAs that share the walk of one (row tile, kv head): enough that all walks together fill the SMs, at most 16, and
// none shorter than kSplitTiles of the longest cache. total G / rows tiles, or one per sequence, are the fewest there are.
int prefill_splits(int B, int total, int G, const kda_kv_cache *c) {
    const int R = tile_rows(c->head_dim);
    const long long fewest = std::max<long long>(std::min(B, total), (static_cast<long long>(total) * G + R - 1) / R);
    const long long tiles = (static_cast<long long>(c->max_pages) * c->page_size + kKeys - 1) / kKeys;
    const long long room = static_cast<long long>(num_sms()) * (R == 128 ? 2 : 1);
    return static_cast<int>(std::max<long long>(1, std::min<long long>({16, room / (fewest * c->kv_heads), tiles / kSplitTiles})));
}

// 2-D map over a layer's pool as rows of D values; boxes of 64 channels x min(page, 128) rows.
int make_pool_map(CUtensorMap *tm, const void *base, const KvView &c, int D) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return KDA_ERR_CUDA;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(c.num_pages) * c.kv_heads * c.page_size};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(std::min(c.page_size, kKeys))};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? KDA_OK : KDA_ERR_INVALID_ARG;
}

template <int D>
int launch_prefill(const PrefillArgs &a, unsigned grid, cudaStream_t s) {
    static std::atomic<unsigned long long> attr{0};
    KDA_TRY(smem_opt_in(prefill_kernel<D>, PrefillCfg<D>::BYTES, attr));
    // CTAs beyond the tiles' only look sequences over, 32 each (a loop there made the softmax warps spill)
    const unsigned ctas = std::max(grid * a.splits, static_cast<unsigned>((a.B + 31LL) / 32));
    prefill_kernel<D><<<ctas, PrefillCfg<D>::THREADS, PrefillCfg<D>::BYTES, s>>>(a);
    KDA_TRY(launch_status());
    if (a.splits == 1) return KDA_OK;
    return launch_after(prefill_join_kernel<D>, dim3(grid, tile_rows(D) / 8), dim3(256), 0, s, a);
}

}  // namespace
}  // namespace kda

namespace kda {

namespace {
// Slots of row tiles (see locate): no more than twice what total rows need, however many sequences have none
long long tile_slots(int B, int total, int G, int D) {
    return static_cast<long long>(total) * G / tile_rows(D) + std::min(B, total);
}
}  // namespace

bool attn_tiles_fits(int B, int total, int heads, const kda_kv_cache *cache) {
    const int G = heads / cache->kv_heads;
    return static_cast<long long>(total) * G <= 0x7fffffffLL - 256 &&
           16 * tile_slots(B, total, G, cache->head_dim) * cache->kv_heads <= 0x7fffffffLL;
}

size_t attn_tiles_scratch_bytes(int B, int total, int heads, const kda_kv_cache *cache) {
    const int G = heads / cache->kv_heads, splits = prefill_splits(B, total, G, cache);
    if (splits == 1) return 0;
    const size_t slots = static_cast<size_t>(tile_slots(B, total, G, cache->head_dim));
    return slots * cache->kv_heads * splits * tile_rows(cache->head_dim) * (cache->head_dim + 4) * sizeof(float);
}

int attn_tiles(const kda_kv_cache *cache, int layer, const uint16_t *q, const int *cu, const int *slots, int B,
               int max_rows, int total, int window, int sinks, uint16_t *out, float *lse, void *scratch,
               const kda_dims *dims, cudaStream_t s) {
    PrefillArgs a{};
    const int D = cache->head_dim;
    a.G = dims->heads / cache->kv_heads;
    a.nslots = static_cast<int>(tile_slots(B, total, a.G, D));
    a.splits = prefill_splits(B, total, a.G, cache);
    a.status = device_status_ptr();
    if (!a.status) return KDA_ERR_CUDA;
    a.c = kv_view(cache, layer);
    KDA_TRY(make_pool_map(&a.tk, a.c.k, a.c, D));
    KDA_TRY(make_pool_map(&a.tv, a.c.v, a.c, D));
    a.q = q;
    a.cu = cu;
    a.slots = slots;
    a.out = out;
    a.lse = lse;
    a.B = B;
    a.max_rows = max_rows;
    a.total = total;
    a.heads = dims->heads;
    // a window that holds the longest sequence is none
    a.window = window < a.c.max_pages * a.c.page_size ? window : 0;
    a.sinks = std::min(sinks, a.c.max_pages * a.c.page_size);
    // a negative scale is taken as negated queries, and 0 as one so small that every weight is 1
    a.scale2 = std::max(std::fabs(dims->scale) * 1.4426950408889634f, 1e-30f);
    a.flip = dims->scale < 0.f ? 0x80008000u : 0u;
    a.part_o = static_cast<float *>(scratch);
    a.part_ml = a.part_o + static_cast<size_t>(a.nslots) * cache->kv_heads * a.splits * tile_rows(D) * D;
    const unsigned grid = static_cast<unsigned>(static_cast<long long>(a.nslots) * cache->kv_heads);
    return D == 128 ? launch_prefill<128>(a, grid, s) : launch_prefill<64>(a, grid, s);
}

namespace {

int check_prefill(int B, int max_rows, int total, const kda_dims *dims, const kda_kv_cache *cache) {
    KDA_TRY(check_cache(cache));
    KDA_TRY(check_dims(dims));
    if (B < 0 || max_rows < 0 || total < 0) return KDA_ERR_INVALID_ARG;
    if (dims->head_dim != cache->head_dim || dims->heads % cache->kv_heads) return KDA_ERR_INVALID_ARG;
    if (B > 65535 || dims->heads > 65535) return KDA_ERR_UNSUPPORTED;
    return attn_tiles_fits(B, total, dims->heads, cache) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_attn_prefill_scratch_bytes(int B, int max_rows, int total_tokens, const kda_dims *dims,
                                      const kda_kv_cache *cache) {
    if (kda::check_prefill(B, max_rows, total_tokens, dims, cache) != KDA_OK || B == 0 || total_tokens == 0 || max_rows == 0)
        return 0;
    if (kda::few_rows(max_rows, dims->heads, cache)) return kda::attn_rows_scratch_bytes(max_rows, dims->heads, cache);
    return kda::attn_tiles_scratch_bytes(B, total_tokens, dims->heads, cache);
}

int kda_attn_prefill(const kda_kv_cache *cache, int layer, const kda_bf16 *q, const int *cu_seqlens, const int *slots,
                     int B, int max_rows, int total_tokens, int window, int sinks, kda_bf16 *out, float *lse,
                     void *scratch, size_t scratch_bytes, const kda_dims *dims, void *stream) {
    KDA_TRY(kda::check_prefill(B, max_rows, total_tokens, dims, cache));
    if (!q || !cu_seqlens || !out || window < 0 || sinks < 0 || layer < 0 || layer >= cache->layers)
        return KDA_ERR_INVALID_ARG;
    if (!kda::aligned16(q) || !kda::aligned16(out)) return KDA_ERR_MISALIGNED;
    if (B == 0 || total_tokens == 0) return KDA_OK;
    if (max_rows == 0) return KDA_ERR_INVALID_ARG;
    const size_t need = kda_attn_prefill_scratch_bytes(B, max_rows, total_tokens, dims, cache);
    KDA_TRY(kda::check_scratch(scratch, scratch_bytes, need));
    auto s = static_cast<cudaStream_t>(stream);
    if (kda::few_rows(max_rows, dims->heads, cache))
        return kda::attn_rows(cache, layer, q, cu_seqlens, slots, B, max_rows, total_tokens, window, sinks, out, lse,
                              scratch, dims, s);
    return kda::attn_tiles(cache, layer, q, cu_seqlens, slots, B, max_rows, total_tokens, window, sinks, out, lse,
                           scratch, dims, s);
}

}  // extern "C"
