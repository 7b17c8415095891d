// grouped_gemm.cu -- products of 16-bit rows sorted by expert with their expert's weights, and
// their gradients, on the tcgen05 tensor cores.
//
// Rows [rows][K] are grouped by offsets, as the token plan gives them.  For the rows r of expert e
//   plain       y[r] = x[r] W[e]  (W [E][K][N]),  or x[r] W[e]^T  (W [E][N][K]),  or the sum of
//               two such products of the two halves of x[r] with weights of their own;
//   gated       g = x[r] Wg[e], u = x[r] Wu[e]: p = SiLU(g) u, and g and u in 8 bits;
//   gated grad  q = d[r] Wd[e]^T is the gradient of p; with s = 1 / (1 + e^-g), g and u from 8 bits:
//               dg = q u s (1 + g (1 - s)), du = q g s, and p again;
//   weights     G[e] = sum_r x[r]^T d[r], a product summed over the expert's rows.
// Operands bf16 or f16, sums in the tensor core's fp32 accumulators in the order of K (or of the
// rows), long ones split at fixed places, each result rounded once: a row's result does not depend on
// its group, tile or grid.
//
// A unit is a row tile of one expert times a tile of channels.  The channels are the MMA's M side
// and the rows its N side: N is a group's own number of rows, rounded up to 16 a CTA, so a
// group of 300 rows costs 320, not 384 or 512, and a group's tiles are of equal size.
// Groups need no padding: a copy may run into the next expert's rows, whose results are dropped
// by the epilogue (a row only reaches its own results).  In a weights' gradient rows are what is
// summed: the last rows of the last step are zeroed in shared memory before the MMA reads them.
// The tensor core's accumulators truncate: a chain of n MMAs is off by about n 2^-24 (all addends of one
// sign: f16 twice that).  So an accumulator sums a bounded chain, and those of a longer sum are added up
// in registers, with rounding, at fixed places of K or of the rows.  Chains are
//   8192 of K or rows for 16-bit results: 2^-15, a sixteenth of f16's half step;
//   256 of K for fp32 results (random values, K = 2048: 3.5e-7 off in the 2-norm for 2.5e-6, torch's fp32
//   product 4e-7; 512: 6.5e-7), at 8192 tokens and K = 2048 175 us in place of 166, K = 768 245 of 205,
//   65536 x 2048 x 2048 325 of 290;
//   256 of K for the codes of f16 rows, which a gradient in f16 sees: with codes next to a border on the
//   other side, what is computed from them was up to twice as far off as from fp32 sums (H = 2048,
//   int8: 4.5e-4 for 2.2e-4, now 2.3e-4).  4096 tokens 220 us in place of 185, 8192 tokens 407 of 299: a
//   unit's codes are made while the next unit's first chain runs, no longer the whole unit.  bf16's
//   rounding, 1.7e-3, hides it: bf16 rows are not split;
//   256 rows for an fp32 gradient of weights (8192 tokens 2.2e-7 off in the 2-norm, torch's fp32 products
//   2.7e-7; 512 rows 4.3e-7, one chain 1.1e-6; 241, 232 and 230 us).
//
// Large tile: two CTAs share a tile (cta_group::2): 256 channels, 128 each, times up to 256
// rows, each CTA holding half of the rows' operand: 32 KB of shared memory a stage of 64 of K, so
// a stage's copies are 62 bytes a cycle of its MMAs (one CTA's 128 x 256 takes 94).  Small tile, for
// few rows a group: one CTA, 128 channels (gated: 64 of each projection), up to 16 rows.
//
// Per CTA (persistent, one an SM) 13 warps: 0-3 and 4-7 drain every other 16 rows (weights: 32
// columns) of an accumulator, 8 and 9 issue the copies of the M and N sides, 10 the MMAs (the pair's
// first CTA for both), 11 zeroes the last rows of a weights' gradient, 12 works out the units.  The
// accumulators are double-buffered.  An epilogue warp has 32 channels in its lanes; where a lane
// needs channels of one row, 16 rows of them are turned round through shared memory.
//
// What bounds it, on a GB300 (H = 2048, I = 768, 128 experts, top 8, bf16, groups as a router makes
// them, 7 to 4104 rows at 8192 tokens):
//   one group  65536 rows, K = N = 2048: 315 us, 1.75 PFLOP/s (the library's product: 308); K = 768: 132
//              us (121); 16384 x 8192 x 8192: 1.18 ms (1.05 to 1.28).  MMAs, and the power they take.
//   8192       gate and up 270 us, 1.52 PFLOP/s and 4.3 TB/s; down 155 us, 1.33 PFLOP/s and 5.0 TB/s;
//   tokens     weights' gradient in fp32 241 us, 4.9 TB/s.  The weights' first way from HBM and the MMAs
//              both: groups of under 215 rows take longer to copy than to multiply, and equal groups of
//              512 rows take 245 and 137 us.
//   4096       with the checkpoint 185 us, down's gradient through the gate 130 us, 1.04 and 0.74 GB: HBM,
//   tokens     0.83 of the copy rate.
//   21 tokens  gate and up 68 us for 447 MB, 0.97 of the copy rate.  One token 13 us for 50 MB, down 8.8
//              us for 25 MB: start-up, and 96 to 128 CTAs with 16 KB copies.
#include <string.h>

#include "checkpoint.cuh"
#include "gemm_core.cuh"
#include "grouped.cuh"
#include "row_io.cuh"

namespace moe {

constexpr int kGgWarps = 13;           // 16 where several accumulators are added up, their registers shared out (below)
constexpr int kGgStaging = 3 * 1024;   // a warp's: 16 rows of 32 fp32 channels, and 16 of 16 bits
constexpr int kGgMaxStages = 6;
constexpr int kGgSort = 512;           // weights: rows up to which experts keep their order
constexpr int kGgUnits = 8;            // units that are worked out ahead

template <int kCtas_, int kRows_, int kK_, int kStages_>
struct GgTile {
    static constexpr int kCtas = kCtas_, kRows = kRows_, kStages = kStages_;
    static constexpr int kK = kK_;                   // K per stage
    static constexpr int kChunks = kK / 64;          // K-major: copies of 64 of K
    static constexpr int kCh = 128 * kCtas;          // channels of a unit
    static constexpr int kGran = 16 * kCtas;         // N is a multiple of this
    static constexpr int kSide = kRows / kCtas;      // rows of the N side a CTA holds
    static constexpr int kABytes = 128 * kK * 2;
    static constexpr int kBBytes = kSide * kK * 2;
    static constexpr int kMajor = kK * 128;          // channel-major: a copy of 64 channels
    static constexpr int kAChunk = 128 * 128, kBChunk = kSide * 128;
    static constexpr int kPiece = kCtas == 1 ? kRows : 32;  // rows of a small copy of the N side
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr uint32_t kTmemCols = 2 * kRows;
    static constexpr size_t kSmem = (size_t)kStages * kStageBytes + 8 * kGgStaging + 1024;
    static_assert((kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols >= 32 && kTmemCols <= 512, "tensor memory");
    static_assert(kStageBytes % 1024 == 0 && kBChunk % 1024 == 0 && kStages <= kGgMaxStages, "stage alignment");
};
using GgLarge = GgTile<2, 256, 64, 6>;
using GgSmall = GgTile<1, 16, 128, 5>;

// A unit, as every role reads it.
struct alignas(16) GgUnit {
    int32_t row0, nrows;  // the row tile's (weights: the expert's) first row and number of rows; < 0: none is left
    int32_t n;            // the MMA's N
    int32_t n0;           // weights: first column
    int32_t e, ct;        // expert, channel tile
    int32_t single;       // the expert has no other row tile
    int32_t unused;
    // weights: the last step's rows past the group's end are zeroed before the MMA reads them
    __device__ __forceinline__ bool ragged() const { return nrows % 16 != 0; }
};

__host__ __device__ constexpr bool gg_sums(Grouped m) { return m == Grouped::kWeights || m == Grouped::kWeights32; }
// Whether the epilogue's warps add up several accumulators, of up to 256 rows or columns, and so get more
// registers than the others.
template <typename G>
__host__ __device__ constexpr bool gg_shares(Grouped m, bool split) {
    return gg_sums(m) || (split && G::kRows > 32);
}
__host__ __device__ constexpr int gg_threads(bool shares) { return 32 * (shares ? 16 : kGgWarps); }
// Weights: rows that one accumulator sums.
__host__ __device__ constexpr int gg_chain(Grouped m) { return m == Grouped::kWeights32 ? 256 : 8192; }
// Products: the K that one accumulator sums, for fp32 results and f16 rows' codes, and for other results.
constexpr int kGgChainFine = 256, kGgChain = 8192;

struct GgCtl {
    GgUnit units[kGgUnits];
    uint64_t ufull[kGgUnits];
    uint64_t uempty[kGgUnits];     // all roles have read the unit
    uint64_t full[kGgMaxStages];   // the pair's first CTA: both CTAs' copies of a stage
    uint64_t empty[kGgMaxStages];
    uint64_t land[kGgMaxStages];   // weights: copies of a stage whose last rows are to be zeroed
    uint64_t tfull[2];
    uint64_t tempty[2];            // the pair's first CTA: all epilogue warps of both
    uint64_t done;
    uint32_t tmem;
    volatile int abort;
    int32_t wsum[16];
    int32_t first_row, valid_rows;  // of all groups
    alignas(16) int32_t first[kGroupedMaxExperts + 4];  // row tiles before expert e; weights: its rows
    uint16_t order[kGroupedMaxExperts];     // rows of expert e's tiles; weights: experts, those of most rows first
};

// x, x2: the rows' boxes are a CTA's side, and of the small ones (xs, x2s) 32 rows.  Weights: x the
// rows, w the grads; xs, x2s the same in chunks of 64 channels, two a box.
struct GgMaps {
    CUtensorMap x, x2, xs, x2s, w, w2, y, p;
};

struct GgArgs {
    const int32_t *offsets;
    int64_t rows;
    int E, C, K, N;   // C channels; N the weights' gradient's columns
    int parts, nct, nnt;
    int chain, pieces;   // split: the K of an accumulator, a unit's accumulators
    int deep_m, deep_n;  // the M, N side's channels are whole chunks of 64: one copy brings two
    int dt, dct;      // a step of a CTA pair's units in row tiles and channel tiles
    uint32_t idesc;   // without N
    int half, out32;  // f16 (else bf16) results; fp32 ones
    int bulk;         // kPlain: y allows tensor stores
    int vec;          // rows of out allow stores of 32, 16 bytes or elements: 2, 1, 0
    unsigned char *out;
    int64_t ldo;
    unsigned char *p;
    int pvec;
    int code, pitch;
    uint8_t *codes, *scales;
    int32_t *status;
};

// ---------------------------------------------------------------------- pairs of CTAs (PTX)
// Address, in the cluster's window, of the pair's first CTA's copy of a barrier.
template <int kCtas>
__device__ __forceinline__ uint32_t gg_leader(uint64_t *bar) {
    if constexpr (kCtas == 1) return smem_u32(bar);
    else return map_shared_rank(bar, 0);
}
// (At the scope of the CTA: what the thread has written before is not what a waiter in the other CTA
// reads.  With release at cluster scope in the producers too, every stage waited a memory barrier
// out, 0.75 us, and products ran at half the rate.)
__device__ __forceinline__ void gg_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// What the thread has written to shared memory is visible to whoever waits for the barrier.
__device__ __forceinline__ void gg_arrive_release(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// Waits take a barrier's shared-memory address.  kCluster: what the other CTA's thread wrote before
// its releasing arrival is visible after.
template <bool kCluster>
__device__ __forceinline__ bool gg_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (kCluster)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    return ok != 0;
}
// Bounded.  What follows the first tries is kept out of the loops that wait, whose instructions a
// single thread fetches anew every time.
template <bool kCluster>
__device__ __noinline__ bool gg_wait_slow(uint32_t bar, uint32_t parity, GgCtl *ctl) {
    const uint64_t t0 = globaltimer_ns();
    while (!gg_try<kCluster>(bar, parity)) {
        if (ctl->abort) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            ctl->abort = 1;
            return false;
        }
    }
    return true;
}
// kInline: without a call, for kernels whose warps share their registers out.
template <bool kCluster = false, bool kInline = false>
__device__ __forceinline__ bool gg_wait_one(uint32_t bar, uint32_t parity, GgCtl &ctl) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
        if (gg_try<kCluster>(bar, parity)) return true;
    if constexpr (!kInline) return gg_wait_slow<kCluster>(bar, parity, &ctl);
    const uint64_t t0 = globaltimer_ns();
    while (!gg_try<kCluster>(bar, parity)) {
        if (!ctl.abort && globaltimer_ns() - t0 > kWaitLimitNs) ctl.abort = 1;
        if (ctl.abort) return false;
    }
    return true;
}
// The same for a whole warp, with one answer.
template <bool kInline = false>
__device__ __forceinline__ bool gg_wait(uint64_t *bar, uint32_t parity, GgCtl &ctl) {
    return __all_sync(0xffffffffu, gg_wait_one<false, kInline>(smem_u32(bar), parity, ctl));
}
// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool gg_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

template <int kCtas>
__device__ __forceinline__ void gg_load_2d(uint32_t dst, const CUtensorMap *tm, int x, int y, uint32_t bar, uint64_t policy) {
    if constexpr (kCtas == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar), "l"(policy)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint "
            "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar), "l"(policy)
            : "memory");
}
template <int kCtas>
__device__ __forceinline__ void gg_load_3d(uint32_t dst, const CUtensorMap *tm, int x, int y, int z, uint32_t bar,
                                           uint64_t policy) {
    if constexpr (kCtas == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint "
            "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
            : "memory");
}

template <int kCtas>
__device__ __forceinline__ void gg_load_4d(uint32_t dst, const CUtensorMap *tm, int x, int y, int z, int w, uint32_t bar,
                                           uint64_t policy) {
    if constexpr (kCtas == 1)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint "
            "[%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
            : "memory");
}

template <int kCtas>
__device__ __forceinline__ void gg_mma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, bool accumulate) {
    if constexpr (kCtas == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"((uint32_t)accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"((uint32_t)accumulate)
            : "memory");
}
// Arrives on the barrier, in both CTAs of a pair, when all MMAs issued so far are complete.
template <int kCtas>
__device__ __forceinline__ void gg_commit(uint64_t *bar) {
    if constexpr (kCtas == 1) umma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
}
template <int kCtas>
__device__ __forceinline__ void gg_tmem_alloc(uint32_t *slot, uint32_t cols) {
    if constexpr (kCtas == 1) tmem_alloc(slot, cols);
    else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int kCtas>
__device__ __forceinline__ void gg_tmem_dealloc(uint32_t tmem, uint32_t cols) {
    if constexpr (kCtas == 1) tmem_dealloc(tmem, cols);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}

// ------------------------------------------------------------------------------------ units
// Rows [lo, hi) of expert e; offsets outside [0, rows] or running backwards are clamped.
__device__ __forceinline__ void gg_span(const GgArgs &a, int e, int &lo, int &hi) {
    int64_t b = 0, c = a.rows;
    if (a.offsets) b = a.offsets[e], c = a.offsets[e + 1];
    b = b < 0 ? 0 : (b > a.rows ? a.rows : b);
    c = c < b ? b : (c > a.rows ? a.rows : c);
    lo = (int)b, hi = (int)c;
}

// One warp works the units out and puts them into a ring that the other roles read: where each role
// worked them out itself, the code that a unit begins with, which no warp had run for thousands of
// cycles, kept the MMAs from their next unit for 1450 cycles.
//
// A pair's units.  Products: u = its number, + the number of pairs, ...; unit u is channel tile u % nct
// of row tile u / nct.  Weights: unit u is channel tile u % nct, column tile (u / nct) % nnt of the
// expert with the (u / nct / nnt)-th most rows, and the pairs take them there and back: what one
// takes before another in one turn it takes after it in the next.
template <Grouped kMode, typename G, bool kInline>
__device__ __forceinline__ void gg_schedule(const GgArgs &a, GgCtl &ctl, int tiles) {
    constexpr bool kWeights = gg_sums(kMode);
    const int lane = threadIdx.x & 31, pair = blockIdx.x / G::kCtas, pairs = gridDim.x / G::kCtas;
    int t = pair / a.nct, ct = pair % a.nct, e = 0;
    for (uint32_t turn = 0;; ++turn) {
        GgUnit x;
        x.nrows = -1, x.row0 = x.n = x.n0 = x.e = x.ct = x.single = x.unused = 0;
        if (kWeights) {
            const int64_t u = (int64_t)turn * pairs + ((turn & 1) ? pairs - 1 - pair : pair);
            if (u < (int64_t)a.E * a.nnt * a.nct) {
                const int c = (int)u / a.nct, at = c / a.nnt;
                x.e = ctl.order[at], x.ct = (int)u - c * a.nct, x.n0 = (c - at * a.nnt) * G::kRows;
                int hi;
                gg_span(a, x.e, x.row0, hi);
                x.nrows = ctl.first[x.e];
                x.n = a.N - x.n0 < G::kRows ? a.N - x.n0 : G::kRows;
            }
        } else if (t < tiles) {
            unsigned past;
            do {  // the next expert with the warp's 32 lanes at once
                const int i = e + 1 + lane;
                past = __ballot_sync(0xffffffffu, i <= a.E && ctl.first[i] <= t);
                e += __popc(past);
            } while (past == 0xffffffffu);
            const int q = ctl.order[e];  // rows of a tile
            int lo, hi;
            gg_span(a, e, lo, hi);
            x.row0 = lo + (t - ctl.first[e]) * q;
            x.n = x.nrows = hi - x.row0 < q ? hi - x.row0 : q;
            x.e = e, x.ct = ct, x.single = ctl.first[e + 1] - ctl.first[e] == 1;
            t += a.dt, ct += a.dct;
            if (ct >= a.nct) ct -= a.nct, ++t;
        }
        x.n = (x.n + G::kGran - 1) / G::kGran * G::kGran;
        const uint32_t slot = turn % kGgUnits;
        if (!gg_wait<kInline>(&ctl.uempty[slot], ((turn / kGgUnits) & 1u) ^ 1u, ctl)) return;
        if (lane == 0) {
            ctl.units[slot] = x;
            mbar_arrive(&ctl.ufull[slot]);
        }
        __syncwarp();
        if (x.nrows < 0) return;
    }
}

// The next unit, for a whole warp or for one thread; false when none is left or a wait gave up.
template <bool kWarp, bool kInline = false>
__device__ __forceinline__ bool gg_next(GgCtl &ctl, uint32_t &at, GgUnit &x) {
    const uint32_t slot = at % kGgUnits, parity = (at / kGgUnits) & 1u;
    ++at;
    if (!(kWarp ? gg_wait<kInline>(&ctl.ufull[slot], parity, ctl) : gg_wait_one<false, kInline>(smem_u32(&ctl.ufull[slot]), parity, ctl))) return false;
    x = ctl.units[slot];
    if (kWarp) __syncwarp();
    if (!kWarp || (threadIdx.x & 31) == 0) mbar_arrive(&ctl.uempty[slot]);
    return x.nrows >= 0;
}

// ------------------------------------------------------------------------------- split sums
// kN blocks of 16 columns, 32 apart, by one wait.
template <int kN>
__device__ __forceinline__ void gg_read(uint32_t d, uint32_t (&r)[kN][16]) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[i][0]), "=r"(r[i][1]), "=r"(r[i][2]), "=r"(r[i][3]), "=r"(r[i][4]), "=r"(r[i][5]), "=r"(r[i][6]),
              "=r"(r[i][7]), "=r"(r[i][8]), "=r"(r[i][9]), "=r"(r[i][10]), "=r"(r[i][11]), "=r"(r[i][12]), "=r"(r[i][13]),
              "=r"(r[i][14]), "=r"(r[i][15])
            : "r"(d + 32 * i));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    // (operands, so that no use of them moves above the wait)
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < 16; j += 8)
            asm volatile("" : "+r"(r[i][j]), "+r"(r[i][j + 1]), "+r"(r[i][j + 2]), "+r"(r[i][j + 3]), "+r"(r[i][j + 4]),
                              "+r"(r[i][j + 5]), "+r"(r[i][j + 6]), "+r"(r[i][j + 7]));
}

// -------------------------------------------------------------------------------- epilogues
__device__ __forceinline__ uint32_t gg_pack(float lo, float hi, int half) {
    return half ? pack2<__half>(lo, hi) : pack2<__nv_bfloat16>(lo, hi);
}

// kWords words of a row, by stores of 32 or 16 bytes (vec 2, 1) or as 16-bit elements; `words` of
// them lie within the row.
template <int kWords>
__device__ __forceinline__ void gg_put(unsigned char *dst, const uint32_t (&o)[kWords], int words, int vec) {
    if (vec == 2 && words == kWords && kWords % 8 == 0) {
#pragma unroll
        for (int i = 0; i + 8 <= kWords; i += 8) st_global_32(dst + 4 * i, &o[i]);
    } else if (vec) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
            if (i + 4 <= words) *reinterpret_cast<uint4 *>(dst + 4 * i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if (i < words) {
                reinterpret_cast<uint16_t *>(dst)[2 * i] = (uint16_t)o[i];
                reinterpret_cast<uint16_t *>(dst)[2 * i + 1] = (uint16_t)(o[i] >> 16);
            }
    }
}

__device__ __forceinline__ uint32_t gg_pack(uint64_t v, int half) {
    float lo, hi;
    f2_split(v, lo, hi);
    return gg_pack(lo, hi, half);
}

// s = 1 / (1 + 2^(-g log2 e)) by the approximate power and reciprocal, within 2^-21 (1 + |g| / 4) of
// its value for negative g, 2^-21 for others: what follows is rounded to 16 bits.  Below g = -87.3
// the reciprocal is 0, for values under 2^-119.
__device__ __forceinline__ uint64_t gg_sigmoid(uint64_t g) {
    constexpr float k = -1.4426950408889634f;
    float a, b;
    f2_split(f2_mul(g, f2(k, k)), a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    f2_split(f2_add(f2(a, b), f2(1.0f, 1.0f)), a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return f2(a, b);
}

// Sixteen 16-bit results to a row.
__device__ __forceinline__ void gg_put16(unsigned char *dst, const uint64_t (&v)[8], int half, int vec) {
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = gg_pack(v[i], half);
    gg_put(dst, o, 8, vec);
}

// Lane's channel of 16 rows in, channels of a row out.  Rows are 128 bytes, their 16-byte pieces
// exchanged as a tensor store's 128-byte swizzle has them: no bank conflicts either way.
__device__ __forceinline__ void gg_turn_write(float *turn, int lane, const float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) turn[i * 32 + (lane ^ (4 * (i & 7)))] = v[i];
}
template <int kN>
__device__ __forceinline__ void gg_turn_read(const float *turn, int row, int at, float (&v)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(turn + row * 32 + ((((at + i) >> 2) ^ (row & 7)) << 2));
        v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
    }
}
template <int kN>
__device__ __forceinline__ void gg_turn_read(const float *turn, int row, int at, uint64_t (&v)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(turn + row * 32 + ((((at + 2 * i) >> 2) ^ (row & 7)) << 2));
        v[i] = f.x, v[i + 1] = f.y;
    }
}

// 16 rows of 64 bytes (128 bytes of fp32) by a tensor store through a warp's staging memory, whose
// 16-byte pieces are exchanged as the map's swizzle has them.  (Lanes' own stores of 32 bytes a row
// took 7000 cycles a unit of 256 rows, more than the MMAs of K = 768.)  x: bytes along the row.
__device__ __forceinline__ void gg_store(const CUtensorMap &tm, const void *staging, int x, int row, int lane) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0)
        asm volatile(
            "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\t"
            "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(&tm)),
            "r"(x), "r"(row), "r"(smem_u32(staging))
            : "memory");
}
// All but the last kLeft of this thread's stores have read their staging memory.
template <int kLeft>
__device__ __forceinline__ void gg_store_wait(int lane) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
    __syncwarp();
}
// Sixteen 16-bit results of row lane % 16, from channel 16 (lane / 16), to staging.
__device__ __forceinline__ void gg_stage16(unsigned char *staging, int lane, const uint64_t (&v)[8], int half) {
    const int r = lane & 15, h = lane >> 4;
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = gg_pack(v[i], half);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint4 *>(staging + r * 64 + (((2 * h + i) ^ ((r >> 1) & 3)) << 4)) =
            make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
}

template <typename G>
__device__ __forceinline__ void gg_plain(const GgArgs &a, const CUtensorMap &tm, float *turn, uint32_t d, int lane, int group,
                                         int row0, int nrows, int ch0, uint32_t &turns) {
    const int r = lane & 15, ch = ch0 + 16 * (lane >> 4);
    const int left = a.C - ch, elem = a.out32 ? 4 : 2;
    unsigned char *dst = a.out + ((int64_t)row0 * a.ldo + ch) * elem, *const staging = reinterpret_cast<unsigned char *>(turn);
#pragma unroll 1
    for (int c = 16 * group; c < nrows; c += 32) {
        float v[16];
        if (a.bulk && c + 16 <= nrows) {
            if (a.out32) {
                gg_store_wait<0>(lane);
                tmem_ld16(d + c, v);
                gg_turn_write(turn, lane, v);
                gg_store(tm, staging, ch0 * 4, row0 + c, lane);
            } else {
                unsigned char *const at = staging + 1024 * (turns++ & 1u);  // (counted over all units)
                gg_store_wait<1>(lane);
                tmem_ld16(d + c, v);
                // the lane's channel, as 16 bits, of 16 rows
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const uint32_t two = gg_pack(v[i], v[i + 1], a.half);
                    unsigned char *const to = at + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2;
                    *reinterpret_cast<uint16_t *>(to) = (uint16_t)two;
                    *reinterpret_cast<uint16_t *>(to + 64) = (uint16_t)(two >> 16);
                }
                gg_store(tm, at, ch0 * 2, row0 + c, lane);
            }
            continue;
        }
        // the tile's last rows: no row behind them is written
        gg_store_wait<0>(lane);
        tmem_ld16(d + c, v);
        gg_turn_write(turn, lane, v);
        __syncwarp();
        gg_turn_read(turn, r, 16 * (lane >> 4), v);
        if (c + r < nrows && left > 0) {
            unsigned char *at = dst + (int64_t)(c + r) * a.ldo * elem;
            if (a.out32) {
                uint32_t o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(v[i]);
                gg_put(at, o, left < 16 ? left : 16, a.vec);
            } else {
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = gg_pack(v[2 * i], v[2 * i + 1], a.half);
                gg_put(at, o, left < 16 ? left / 2 : 8, a.vec);
            }
        }
        __syncwarp();
    }
}

// Sixteen values of this lane and its neighbour's (lane ^ 16) as a block of the checkpoint.
template <bool kInt8>
__device__ __forceinline__ void gg_block(const GgArgs &a, const float (&v)[16], int64_t row, int col, int lane, bool live) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) top = max_abs(top, v[i], v[i + 1]);
    const uint32_t mine = __float_as_uint(top) & 0x7fffffffu, other = __shfl_xor_sync(0xffffffffu, mine, 16);
    const uint32_t byte = eight_byte<kInt8>(other > mine ? other : mine);
    const uint4 code = eight_codes<kInt8>(v, byte);
    if (!live) return;
    *reinterpret_cast<uint4 *>(a.codes + row * (2 * a.C) + col + 16 * (lane >> 4)) = code;
    if (lane < 16) a.scales[row * a.pitch + col / 32] = (uint8_t)byte;
}

// Two warps, of 32 gate channels and of the same 32 up channels.  Each quantises its own; p of the
// first 8 of 16 rows is the gate warp's, of the last 8 the up warp's.
__device__ __forceinline__ void gg_gated(const GgArgs &a, float *turn, float *other, uint32_t d, int lane, int group,
                                         int bar, bool up, int row0, int nrows, int ch0) {
    const int r = lane & 15, h = lane >> 4, pr = (lane & 7) + (up ? 8 : 0), pch = 8 * (lane >> 3);
    float *const tg = up ? other : turn, *const tu = up ? turn : other;
    unsigned char *dst = a.out + ((int64_t)row0 * a.ldo + ch0 + pch) * 2;
#pragma unroll 1
    for (int c = 16 * group; c < nrows; c += 32) {
        float v[16];
        tmem_ld16(d + c, v);
        named_bar_sync(bar, 64);  // both have read the rows before
        gg_turn_write(turn, lane, v);
        named_bar_sync(bar, 64);
        if (a.codes) {
            gg_turn_read(turn, r, 16 * h, v);
            const int col = (up ? a.C : 0) + ch0;
            const bool live = c + r < nrows;
            if (a.code == MOE_CODE_INT8) gg_block<true>(a, v, (int64_t)row0 + c + r, col, lane, live);
            else gg_block<false>(a, v, (int64_t)row0 + c + r, col, lane, live);
        }
        uint64_t g[4], u[4];
        gg_turn_read(tg, pr, pch, g);
        gg_turn_read(tu, pr, pch, u);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = gg_pack(f2_mul(f2_mul(g[i], gg_sigmoid(g[i])), u[i]), a.half);
        if (c + pr < nrows) gg_put(dst + (int64_t)(c + pr) * a.ldo * 2, o, 4, a.vec);
    }
}

// A lane's part of the checkpoint: sixteen codes and the scale byte of g and of u.
struct GgCodes {
    uint4 g, u;
    uint32_t gs, us;
};
__device__ __forceinline__ GgCodes gg_codes(const GgArgs &a, int64_t row, int ch, bool live) {
    GgCodes c{};
    if (live) {
        const uint8_t *p = a.codes + row * (2 * a.C) + ch, *q = a.scales + row * a.pitch;
        c.g = *reinterpret_cast<const uint4 *>(p), c.u = *reinterpret_cast<const uint4 *>(p + a.C);
        c.gs = q[ch / 32], c.us = q[(a.C + ch) / 32];
    }
    return c;
}

// The checkpoint is read two steps of 16 rows ahead, the first before the unit's sums are complete:
// read where they are used, the codes' way from memory took 3250 cycles a step.
template <bool kInt8>
__device__ __forceinline__ void gg_gated_grad(const GgArgs &a, const GgMaps &tm, float *turn, uint32_t d, int lane, int group, int row0,
                                              int nrows, int ch0, GgCodes (&next)[2]) {
    const int r = lane & 15, h = lane >> 4, ch = ch0 + 16 * h, I = a.C;
#pragma unroll 2
    for (int c = 16 * group; c < nrows; c += 32) {
        const bool live = c + r < nrows;
        const int64_t row = (int64_t)row0 + c + r;
        const GgCodes now = next[0];
        next[0] = next[1];
        next[1] = gg_codes(a, row + 64, ch, c + 64 + r < nrows);
        float v[16];
        uint64_t q[8], g[8], u[8];
        unsigned char *const staging = reinterpret_cast<unsigned char *>(turn);
        tmem_ld16(d + c, v);
        if (a.p) gg_store_wait<1>(lane);  // all but the last store, of p from its own memory
        else gg_store_wait<0>(lane);
        gg_turn_write(turn, lane, v);
        __syncwarp();
        gg_turn_read(turn, r, 16 * h, q);
        eight_values<kInt8>(now.g, now.gs, g);
        eight_values<kInt8>(now.u, now.us, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t s = gg_sigmoid(g[i]), gs = f2_mul(g[i], s), t = f2_mul(q[i], u[i]);
            const uint64_t rest = f2_fma(s, f2(-1.0f, -1.0f), f2(1.0f, 1.0f));
            u[i] = f2_mul(u[i], gs);                       // p
            q[i] = f2_mul(q[i], gs);                       // grad of u
            g[i] = f2_mul(t, f2_fma(gs, rest, s));         // grad of g
        }
        if (c + 16 <= nrows) {
            __syncwarp();
            gg_stage16(staging, lane, g, a.half);
            gg_store(tm.y, staging, ch0 * 2, row0 + c, lane);
            gg_stage16(staging + 1024, lane, q, a.half);
            gg_store(tm.y, staging + 1024, (I + ch0) * 2, row0 + c, lane);
            if (a.p) {
                gg_store_wait<2>(lane);  // the last p
                gg_stage16(staging + 2048, lane, u, a.half);
                gg_store(tm.p, staging + 2048, ch0 * 2, row0 + c, lane);
            }
        } else if (live) {
            unsigned char *dst = a.out + (row * (2 * I) + ch) * 2;
            gg_put16(dst, g, a.half, a.vec);
            gg_put16(dst + 2 * I, q, a.half, a.vec);
            if (a.p) gg_put16(a.p + (row * I + ch) * 2, u, a.half, a.pvec);
        }
        __syncwarp();
    }
}

// A warp's 32 rows of 32 columns of the gradient, by tensor stores of 64-byte rows (clipped at the
// gradient's edges) through its staging memory.
template <bool k32>
__device__ __forceinline__ void gg_weights_put(const GgArgs &a, const CUtensorMap &tm, unsigned char *staging, int lane, int e,
                                               int ch0, int col, const float (&v)[32]) {
#pragma unroll
    for (int q = 0; q < (k32 ? 2 : 1); ++q) {
        gg_store_wait<0>(lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 o;
            if constexpr (k32) {
                o = make_uint4(__float_as_uint(v[16 * q + 4 * i]), __float_as_uint(v[16 * q + 4 * i + 1]),
                               __float_as_uint(v[16 * q + 4 * i + 2]), __float_as_uint(v[16 * q + 4 * i + 3]));
            } else {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = gg_pack(v[8 * i + 2 * j], v[8 * i + 2 * j + 1], a.half);
                o = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<uint4 *>(staging + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) = o;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            asm volatile(
                "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
                "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(&tm)),
                "r"(col * (k32 ? 4 : 2) + 64 * q), "r"(ch0), "r"(e), "r"(smem_u32(staging))
                : "memory");
    }
}

// The warp's part of a unit: every other 32 of its n columns; zeros for an expert without rows.
template <bool k32>
__device__ __forceinline__ void gg_weights(const GgArgs &a, const CUtensorMap &tm, unsigned char *staging, uint32_t d,
                                           int lane, int group, int e, int ch0, int n0, int n, bool zero) {
#pragma unroll 1
    for (int c = 32 * group; c < n && n0 + c < a.N; c += 64) {
        float v[32];
        uint32_t w[32];
        if (!zero) {
            tmem_ld32(d + c, w);
            tmem_ld_wait(w);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = zero ? 0.0f : __uint_as_float(w[i]);
        gg_weights_put<k32>(a, tm, staging, lane, e, ch0, n0 + c, v);
    }
}

// `bytes` (a multiple of 16; of 2 when the address is not 16-byte aligned) of zeros by 128 threads.
__device__ __forceinline__ void gg_zero(unsigned char *p, int64_t bytes, bool wide) {
    if (wide)
        for (int64_t i = 16 * (int64_t)(threadIdx.x & 127); i < bytes; i += 16 * 128)
            *reinterpret_cast<uint4 *>(p + i) = uint4{0, 0, 0, 0};
    else
        for (int64_t i = 2 * (int64_t)(threadIdx.x & 127); i < bytes; i += 2 * 128) *reinterpret_cast<uint16_t *>(p + i) = 0;
}

// -------------------------------------------------------------------------------- producers
// A warp that copies one side's operand (kSideM: the M side's); one lane does, its registers hold the
// ring's state.  What a stage takes between its memory's release and its copies is kept short: with
// the coordinates and addresses worked out there it took 400 cycles, in every turn of the ring.
template <Grouped kMode, bool kTrans, typename G, bool kSideM, bool kInline>
__device__ __forceinline__ void gg_produce(const GgMaps &tm, const GgArgs &a, GgCtl &ctl, uint32_t base, int rank) {
    constexpr bool kWeights = gg_sums(kMode), kGated = kMode == Grouped::kGated;
    constexpr int kCtas = G::kCtas;
    constexpr bool kByK = kSideM ? kTrans : !kWeights;  // copies of 64 of K, else of 64 channels
    constexpr int kChunk = !kByK ? G::kMajor : kSideM ? G::kAChunk : G::kBChunk;
    // Copies of a whole stage in CTA r of the pair; those that bring nothing which the MMAs read, or
    // whose results are stored, are left out.
    auto wide = [&](const GgUnit &x, int r) {
        const int part = kSideM ? 128 : x.n / kCtas;
        const int left = (kSideM ? a.C - (x.ct * kCtas) * (kGated ? 64 : 128) : kWeights ? a.N - x.n0 : x.nrows) -
                         r * (kSideM && kGated ? 64 : part);
        return left <= 0 ? 0 : kByK ? G::kChunks : (kSideM && kGated) || (part > 64 && left > 64) ? 2 : 1;
    };
    // weights that one row tile reads leave L2 first
    const uint64_t keep = policy_evict_normal(), once = policy_evict_first();
    const uint32_t full0 = gg_leader<kCtas>(&ctl.full[0]), own0 = smem_u32(&ctl.full[0]), empty0 = smem_u32(&ctl.empty[0]);
    if (gg_elect()) {
        uint32_t dst = base, slot = 0, parity = 1, it = 0, unit = 0;  // slot: 8 x stage
        bool ok = true;
        GgUnit x;
        while (ok && gg_next<false, kInline>(ctl, unit, x)) {
            const uint64_t pol = !kWeights && kSideM && x.single ? once : keep;
            int n = wide(x, rank), both = kCtas == 1 ? n : wide(x, 0) + wide(x, 1), chunk = kChunk, dx = 128, dy = 0;
            const int part_n = x.n / kCtas;
            if (kByK && !kSideM && part_n <= G::kSide - G::kPiece) {
                // as many copies of 32 rows as the side has, where that is fewer bytes than its whole box
                static_assert(G::kChunks == 1 || G::kSide == G::kPiece, "one chunk of K a stage");
                const int pieces = (part_n + G::kPiece - 1) / G::kPiece;
                n = n ? pieces : 0, both = both * pieces, chunk = G::kPiece * 128, dx = 0, dy = G::kPiece;
            }
            const bool small_box = dy != 0;
            const bool deep = !kByK && !(kSideM && kGated) && (kSideM ? a.deep_m : a.deep_n && part_n % 64 == 0);
            if (deep) both = kCtas == 1 ? n > 0 : (wide(x, 0) > 0) + (wide(x, 1) > 0), n = n > 0, chunk = 2 * kChunk;
            const uint32_t tx = (uint32_t)(both * chunk);
            // coordinates: bytes along the operand's rows, the row (of K, or a row of x or w), the expert
            const int fixed = kSideM ? (x.ct * kCtas + rank) * (kGated ? 64 : 128)
                                     : (kWeights ? x.n0 : x.row0) + rank * part_n;
            const int parts = kWeights ? 1 : a.parts, length = kWeights ? x.nrows : a.K;
            const bool ragged = kWeights && x.ragged();
            for (int part = 0; part < parts && ok; ++part) {
                const CUtensorMap *const m = kSideM ? (kWeights ? (deep ? &tm.xs : &tm.x) : part ? &tm.w2 : &tm.w)
                                             : kWeights  ? (deep ? &tm.x2s : &tm.w)
                                             : small_box ? (part ? &tm.x2s : &tm.xs)
                                                         : (part ? &tm.x2 : &tm.x);
                int cx = kByK ? 0 : 2 * fixed, cy = kByK ? fixed : kWeights ? x.row0 : 0;
                for (int left = length; left > 0; left -= G::kK, ++it) {
                    uint32_t bar = full0 + slot, bytes = tx;
                    int copies = n;
                    if (kByK && G::kChunks > 1 && left < G::kK) {
                        const int deep = (left + 63) / 64;
                        copies = n ? deep : 0, bytes = (uint32_t)(both / G::kChunks * deep * chunk);
                    }
                    if (!(ok = gg_wait_one<false, kInline>(empty0 + slot, parity, ctl))) break;
                    // the pair's first CTA expects both CTAs' bytes; a stage whose last rows are to be
                    // zeroed first is each CTA's own
                    if (kWeights && ragged && left <= G::kK) {
                        uint64_t *const land = &ctl.land[slot / 8];
                        bar = smem_u32(land);
                        mbar_arrive_expect_tx(land, (uint32_t)(n * chunk));
                    } else if (rank == 0) {
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(own0 + slot), "r"(bytes)
                                     : "memory");
                    }
                    if constexpr (kSideM && kGated) {
                        if (copies) {
                            gg_load_3d<kCtas>(dst, m, cx, cy, x.e, bar, pol);
                            gg_load_3d<kCtas>(dst + kChunk, &tm.w2, cx, cy, x.e, bar, pol);
                        }
                    } else if (deep) {
                        if (copies) {
                            if constexpr (kWeights) gg_load_3d<kCtas>(dst, m, 0, cy, fixed / 64, bar, pol);
                            else gg_load_4d<kCtas>(dst, m, 0, cy, fixed / 64, x.e, bar, pol);
                        }
                    } else {
                        int px = cx, py = cy;
                        uint32_t pd = dst;
#pragma unroll 1
                        for (int i = 0; i < copies; ++i, px += dx, py += dy, pd += chunk) {
                            if constexpr (kSideM && !kWeights) gg_load_3d<kCtas>(pd, m, px, py, x.e, bar, pol);
                            else gg_load_2d<kCtas>(pd, m, px, py, bar, pol);
                        }
                    }
                    if (kByK) cx += 2 * G::kK;
                    else cy += G::kK;
                    slot += 8, dst += G::kStageBytes;
                    if (slot == 8 * G::kStages) slot = 0, dst = base, parity ^= 1u;
                }
            }
        }
        // every copy has landed before the CTA can exit (after a wait that gave up; else the MMAs have
        // read them all)
        if (rank == 0)
            for (uint32_t i = 0; i < G::kStages && i < it; ++i) {
                const uint32_t at = it - 1 - i;
                if (!mbar_wait_bounded(&ctl.full[at % G::kStages], (at / G::kStages) & 1u)) ctl.abort = 1;
            }
    }
    __syncwarp();
}

// ----------------------------------------------------------------------------------- kernel
// kTrans: the M side's operand is K-major (weights [channels][K]), else channel-major.  kSplit: a product
// whose units take several accumulators one after the other, of a.chain of K each.
template <Grouped kMode, bool kTrans, typename G, bool kSplit>
__global__ void __launch_bounds__(gg_threads(gg_shares<G>(kMode, kSplit)), 1)
grouped_gemm_kernel(const __grid_constant__ GgMaps tm, const GgArgs a) {
    constexpr bool kWeights = gg_sums(kMode), kGated = kMode == Grouped::kGated;
    constexpr bool kShare = gg_shares<G>(kMode, kSplit);
    constexpr int kCtas = G::kCtas, kThreads = gg_threads(kShare);
    constexpr bool kWide = kMode == Grouped::kWeights32;  // an fp32 gradient
    constexpr int kChain = gg_chain(kMode);
    extern __shared__ unsigned char smem_raw[];
    // the same offset in both CTAs of a pair: their descriptors are the first one's
    unsigned char *stages = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char *turns = stages + G::kStages * G::kStageBytes;
    __shared__ GgCtl ctl;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = kCtas == 1 ? 0 : (int)cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(&ctl.full[s], 2);  // the first CTA's producers, or the zeroing warps
            mbar_init(&ctl.empty[s], 1);
            mbar_init(&ctl.land[s], 2);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl.tfull[b], 1);
            mbar_init(&ctl.tempty[b], 8 * kCtas);
        }
        for (int u = 0; u < kGgUnits; ++u) {
            mbar_init(&ctl.ufull[u], 1);
            // eight epilogue warps, two producers, the first CTA's MMAs, weights: the zeroing warp
            mbar_init(&ctl.uempty[u], 10 + (rank == 0) + kWeights);
        }
        mbar_init(&ctl.done, 1);
        ctl.abort = 0;
        fence_mbar_init();
    }
    if (warp == 10) gg_tmem_alloc<kCtas>(&ctl.tmem, G::kTmemCols);
    if (threadIdx.x == 256) {
        prefetch_tensormap(&tm.w);
        prefetch_tensormap(&tm.x);
    }
    pdl_wait();
    pdl_launch_dependents();

    // row tiles before each expert
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += kThreads) {
        const int e = e0 + threadIdx.x;
        int lo = 0, hi = 0;
        if (e < a.E) gg_span(a, e, lo, hi);
        const int tiles = (hi - lo + G::kRows - 1) / G::kRows;
        int inc = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += t;
        }
        if (lane == 31) ctl.wsum[warp] = inc;
        __syncthreads();
        int off = carry, chunk = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            const int t = ctl.wsum[w];
            if (w < warp) off += t;
            chunk += t;
        }
        if (e < a.E) {
            ctl.first[e] = kWeights ? hi - lo : off + inc - tiles;
            // equal tiles: at most kRows, since a group of T tiles has at most T kRows rows
            if (!kWeights && tiles)
                ctl.order[e] = (uint16_t)((hi - lo + G::kGran * tiles - 1) / (G::kGran * tiles) * G::kGran);
            if (e == a.E - 1) {
                ctl.first[a.E] = off + inc;
                ctl.valid_rows = hi;
            }
            if (e == 0) ctl.first_row = lo;
        }
        carry += chunk;
        __syncthreads();
    }
    if constexpr (kWeights) {
        // Experts of many rows first, so that the pairs' last units are short; those of up to kGgSort
        // rows, whose units take their stores' time whatever their rows, as they lie in memory.
        auto key = [&](int rows) { return rows < kGgSort ? kGgSort : rows; };
        for (int e = threadIdx.x; e < a.E; e += kThreads) {
            const int mine = key(ctl.first[e]);
            int rank = 0;
            for (int i = 0; i < a.E; i += 4) {
                const int4 q = *reinterpret_cast<const int4 *>(&ctl.first[i]);
                auto before = [&](int rows, int at) {
                    const int k = key(rows);
                    return at < a.E && (k > mine || (k == mine && at < e));
                };
                rank += before(q.x, i) + before(q.y, i + 1) + before(q.z, i + 2) + before(q.w, i + 3);
            }
            ctl.order[rank] = (uint16_t)e;
        }
    }
    tc_fence_before();
    if constexpr (kCtas == 1) __syncthreads();
    else cluster_sync();
    tc_fence_after();
    const int tiles = kWeights ? a.E : carry;
    if (warp < 8) {
        // 128 registers a thread at the launch, 200 for the two warpgroups here and 56 for the other two:
        // in all the launch's 65,536
        if constexpr (kShare) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int group = warp >> 2, quad = warp & 3;
        unsigned char *const staging = turns + warp * kGgStaging;
        float *const turn = reinterpret_cast<float *>(staging);
        const int bar = 1 + 2 * group + (quad & 1);  // gated: of the gate and up warps of the same channels
        int local = 0;
        uint32_t unit = 0, stored = 0;
        GgUnit x;
        for (;;) {
            bool more = gg_next<true, kShare>(ctl, unit, x);
            // gated: both warps of a barrier go on or neither, also after a wait that gave up
            if constexpr (kGated) more = !named_bar_or(bar, 64, !more);
            if (!more) break;
            const int c0 = (x.ct * kCtas + rank) * (kGated ? 64 : 128) + 32 * (kGated ? quad & 1 : quad);
            if (kWeights && x.nrows == 0) {
                if (c0 < a.C)
                    gg_weights<kWide>(a, tm.y, staging, 0, lane, group, x.e, c0, x.n0, x.n, true);
                continue;
            }
            if (kWeights && x.nrows > kChain) {
                // The accumulators truncate, so a long chain of MMAs loses what rounded sums keep: kChain
                // rows at a time are added up here, in registers.  The tensor memory is free again
                // before the results are stored.
                float sum[4][32];
#pragma unroll
                for (int i = 0; i < 128; ++i) sum[i / 32][i % 32] = 0.0f;
                bool ok = true;
#pragma unroll 1
                for (int rest = x.nrows; rest > 0; rest -= kChain, ++local) {
                    const int buf = local & 1;
                    if (!(ok = gg_wait<kShare>(&ctl.tfull[buf], (uint32_t)(local >> 1) & 1u, ctl))) break;
                    tc_fence_after();
                    const uint32_t d = ctl.tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(buf * G::kRows) + 32 * group;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (c0 >= a.C || 64 * i + 32 * group >= x.n) continue;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float v[16];
                            tmem_ld16(d + 64 * i + 16 * h, v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[i][16 * h + j] += v[j];
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) gg_arrive(gg_leader<kCtas>(&ctl.tempty[buf]));
                }
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c0 < a.C && 64 * i + 32 * group < x.n && x.n0 + 64 * i + 32 * group < a.N)
                        gg_weights_put<kWide>(a, tm.y, staging, lane, x.e, c0, x.n0 + 64 * i + 32 * group, sum[i]);
                continue;
            }
            GgCodes ahead[2];
            if constexpr (kMode == Grouped::kGatedGrad)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 32 * i + 16 * group + (lane & 15);
                    ahead[i] = gg_codes(a, (int64_t)x.row0 + r, c0 + 16 * (lane >> 4), c0 < a.C && r < x.nrows);
                }
            // A split product's accumulators are added up in registers, all but the last one's tensor memory
            // free again at once; the sums go back into the last one's, from where the results are made.
            // (Made from the registers, eight blocks moved up one by one: f16 codes 4096 tokens 226 against
            // 219 us.  One wait for each 16 columns in place of two: 65536 x 2048 x 2048 347 against 318 us.)
            constexpr int kBlocks = kSplit ? (G::kRows + 31) / 32 : 1, kRead = kBlocks < 2 ? kBlocks : 2;
            float sum[kBlocks][16];
#pragma unroll
            for (int i = 0; i < 16 * kBlocks; ++i) sum[i / 16][i % 16] = 0.0f;
            bool ok = true;
            uint32_t d = 0;
            int buf = 0;
            const int pieces = kSplit ? a.pieces : 1;
#pragma unroll 1
            for (int piece = 0; piece < pieces; ++piece, ++local) {
                buf = local & 1;
                if (!(ok = gg_wait<kShare>(&ctl.tfull[buf], (uint32_t)(local >> 1) & 1u, ctl))) break;
                tc_fence_after();
                d = ctl.tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(buf * G::kRows);
                if constexpr (kSplit) {
#pragma unroll
                    for (int i = 0; i < kBlocks; i += kRead) {
                        if (c0 >= a.C || 32 * i + 16 * group >= x.n) continue;
                        uint32_t v[kRead][16];
                        gg_read(d + 32 * i + 16 * group, v);
#pragma unroll
                        for (int j = 0; j < 16 * kRead; ++j) sum[i + j / 16][j % 16] += __uint_as_float(v[j / 16][j % 16]);
                    }
                    if (piece + 1 < pieces) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) gg_arrive(gg_leader<kCtas>(&ctl.tempty[buf]));
                    }
                }
            }
            if constexpr (kGated) ok = !named_bar_or(bar, 64, !ok);
            if (!ok) break;
            if constexpr (kSplit) {
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) {
                    if (c0 >= a.C || 32 * i + 16 * group >= x.n) continue;
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(sum[i][j]);
                    tmem_st16(d + 32 * i + 16 * group, w);
                }
                tmem_st_wait();
            }
            if (c0 >= a.C) {
                // no channel of this warp's lanes
            } else if constexpr (kMode == Grouped::kPlain) {
                gg_plain<G>(a, tm.y, turn, d, lane, group, x.row0, x.nrows, c0, stored);
            } else if constexpr (kGated) {
                gg_gated(a, turn, reinterpret_cast<float *>(turns + (warp ^ 2) * kGgStaging), d, lane, group, bar, quad >= 2,
                         x.row0, x.nrows, c0);
                if (a.codes && c0 == 0 && quad == 0)  // the scale rows' padding
                    for (int r = 32 * group + lane; r < x.nrows; r += 64)
                        for (int b = a.C / 16; b < a.pitch; ++b) a.scales[((int64_t)x.row0 + r) * a.pitch + b] = 0;
            } else if constexpr (kMode == Grouped::kGatedGrad) {
                if (a.code == MOE_CODE_INT8) gg_gated_grad<true>(a, tm, turn, d, lane, group, x.row0, x.nrows, c0, ahead);
                else gg_gated_grad<false>(a, tm, turn, d, lane, group, x.row0, x.nrows, c0, ahead);
            } else {
                gg_weights<kWide>(a, tm.y, staging, d, lane, group, x.e, c0, x.n0, x.n, false);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) gg_arrive(gg_leader<kCtas>(&ctl.tempty[buf]));
        }
        if (lane == 0) bulk_store_wait<false>();  // stores have left shared memory and are visible
        // rows of no group (past the last: dropped routes): zeros
        if (!kWeights && group == 0)
            for (int64_t i = blockIdx.x; i < ctl.first_row + a.rows - ctl.valid_rows; i += gridDim.x) {
                const int64_t r = i < ctl.first_row ? i : i - ctl.first_row + ctl.valid_rows;
                const int elem = a.out32 ? 4 : 2, width = kMode == Grouped::kGatedGrad ? 2 * a.C : a.C;
                gg_zero(a.out + r * a.ldo * elem, (int64_t)width * elem, a.vec > 0);
                if (kMode == Grouped::kGatedGrad && a.p) gg_zero(a.p + r * a.C * 2, (int64_t)a.C * 2, a.pvec > 0);
                if (kGated && a.codes) {
                    gg_zero(a.codes + r * 2 * a.C, 2 * a.C, true);
                    gg_zero(a.scales + r * a.pitch, a.pitch, true);
                }
            }
    } else {
        if constexpr (kShare) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 8 || warp == 9) {
            if (warp == 8) gg_produce<kMode, kTrans, G, true, kShare>(tm, a, ctl, smem_u32(stages), rank);
            else gg_produce<kMode, kTrans, G, false, kShare>(tm, a, ctl, smem_u32(stages) + G::kABytes, rank);
        } else if (warp == 10) {
            if (rank == 0) {
                // 128-byte swizzle, 8-row atoms 1 KB apart.  K-major: a K step of 16 is 32 bytes, a chunk
                // of 64 of K apart from the next.  Channel-major: a K step is two atoms, and channels
                // 64 apart a chunk.  A step only moves the address field (16-byte units).
                constexpr bool kAMajor = !kTrans, kBMajor = kWeights;  // channel-major operands
                const uint64_t a0 = umma_smem_desc(smem_u32(stages), kAMajor ? G::kMajor : 16, 1024, 2);
                const uint64_t b0 = umma_smem_desc(smem_u32(stages) + G::kABytes, kBMajor ? G::kMajor : 16, 1024, 2);
                const uint32_t full0 = smem_u32(&ctl.full[0]);
                if (gg_elect()) {
                    const int parts = kWeights ? 1 : a.parts, summed = a.K;
                    const uint32_t idesc0 = a.idesc, tmem = ctl.tmem;
                    uint32_t stage = 0, parity = 0, at = 0, unit = 0;
                    bool ok = true;
                    GgUnit x;
                    while (ok && gg_next<false, kShare>(ctl, at, x)) {
                        const int length = kWeights ? x.nrows : summed;
                        if (kWeights && length == 0) continue;
                        const uint32_t idesc = idesc0 | (uint32_t)(x.n >> 3) << 17;
                        // an accumulator sums a chain of a part's K (weights: of the rows), or the whole unit
                        constexpr bool kChained = kWeights || kSplit;
                        const int chain = kWeights ? kChain : a.chain;
                        for (int outer = 0; outer < (kSplit ? parts : 1) && ok; ++outer)
                        for (int rest = length; rest > 0 && ok; rest -= chain) {
                            const int take = kChained && rest > chain ? chain : rest;
                            const uint32_t buf = unit & 1u, tparity = ((unit >> 1) & 1u) ^ 1u;
                            const uint32_t d = tmem + buf * G::kRows;
                            bool first = true;
                            ++unit;
                            ok = gg_wait_one<false, kShare>(smem_u32(&ctl.tempty[buf]), tparity, ctl);
                            tc_fence_after();
                            for (int part = 0; part < (kSplit ? 1 : parts) && ok; ++part)
                                for (int left = take; left > 0; left -= G::kK) {
                                    const uint64_t ad = a0 + stage * (G::kStageBytes >> 4);
                                    const uint64_t bd = b0 + stage * (G::kStageBytes >> 4);
                                    auto step = [&](int ks, bool accumulate) {
                                        gg_mma<kCtas>(d, ad + (kAMajor ? ks * 128 : (ks >> 2) * (G::kAChunk >> 4) + (ks & 3) * 2),
                                                      bd + (kBMajor ? ks * 128 : (ks >> 2) * (G::kBChunk >> 4) + (ks & 3) * 2), idesc,
                                                      accumulate);
                                    };
                                    if (!(ok = gg_wait_one<kWeights && kCtas == 2, kShare>(full0 + 8 * stage, parity, ctl))) break;
                                    tc_fence_after();
                                    step(0, !first);
                                    first = false;
                                    if (left >= G::kK) {
#pragma unroll
                                        for (int ks = 1; ks < G::kK / 16; ++ks) step(ks, true);
                                    } else {
#pragma unroll 1
                                        for (int ks = 1; ks * 16 < left; ++ks) step(ks, true);
                                    }
                                    gg_commit<kCtas>(&ctl.empty[stage]);
                                    if (++stage == G::kStages) stage = 0, parity ^= 1u;
                                }
                            if (ok) gg_commit<kCtas>(&ctl.tfull[buf]);
                            if (!kChained) break;
                        }
                    }
                    // every issued MMA has completed before the CTAs free their tensor memory
                    if constexpr (kCtas == 1) umma_commit(&ctl.done);
                    else
                        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                         smem_u32(&ctl.done))
                                     : "memory");
                    if (!mbar_wait_bounded(&ctl.done, 0)) ctl.abort = 1;
                }
                __syncwarp();
            }
        } else if (warp == 11) {
            if constexpr (kWeights) {
                // rows past the group's end within the last K step, as zeros: both operands, since what is
                // there may be a NaN
                int total = 0;
                uint32_t phase = 0, unit = 0;
                GgUnit x;
                while (gg_next<true, kShare>(ctl, unit, x)) {
                    total += (x.nrows + G::kK - 1) / G::kK;
                    if (!x.ragged()) continue;
                    const int stage = (total - 1) % G::kStages;
                    if (!gg_wait<kShare>(&ctl.land[stage], (phase >> stage) & 1u, ctl)) break;
                    phase ^= 1u << stage;
                    const int from = x.nrows % G::kK, to = (from + 15) / 16 * 16;
                    unsigned char *S = stages + stage * G::kStageBytes;
                    for (int i = lane; i < (to - from) * 32; i += 32) {
                        const int ch = i & 3, at = i >> 2;  // four chunks, 16-byte pieces of their rows
                        *reinterpret_cast<uint4 *>(S + ch * G::kMajor + (from + (at >> 3)) * 128 + (at & 7) * 16) = uint4{0, 0, 0, 0};
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) gg_arrive_release(gg_leader<kCtas>(&ctl.full[stage]), 2 / kCtas);
                }
            }
        } else if (warp == 12) {
            gg_schedule<kMode, G, kShare>(a, ctl, tiles);
        }
    }

    tc_fence_before();
    if constexpr (kCtas == 1) __syncthreads();
    else __syncthreads(), cluster_sync();
    tc_fence_after();
    if (warp == 10) gg_tmem_dealloc<kCtas>(ctl.tmem, G::kTmemCols);
    if (threadIdx.x == 0 && ctl.abort) atomicOr(a.status, MOE_DEV_WAIT_TIMEOUT);
}

// ---------------------------------------------------------------------------------- launcher
template <Grouped kMode, bool kTrans, typename G, bool kSplit = false>
static cudaError_t grouped_as(const GgMaps &tm, GgArgs a, cudaStream_t stream) {
    constexpr int per = kMode == Grouped::kGated ? G::kCh / 2 : G::kCh;
    a.nct = (a.C + per - 1) / per;
    a.nnt = (a.N + G::kRows - 1) / G::kRows;
    const int64_t tiles = gg_sums(kMode) ? (int64_t)a.E * a.nnt : (a.rows < a.E ? a.rows : a.rows / G::kRows + a.E);
    const int64_t units = tiles * a.nct, most = num_sms() / G::kCtas;
    const int64_t pairs = units < 1 ? 1 : (units < most ? units : most);
    a.dt = (int)(pairs / a.nct), a.dct = (int)(pairs % a.nct);
    const auto fn = grouped_gemm_kernel<kMode, kTrans, G, kSplit>;
    cudaError_t err = ensure_smem((const void *)fn, G::kSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)(pairs * G::kCtas)), dim3(gg_threads(gg_shares<G>(kMode, kSplit))), G::kSmem, stream, attrs,
                                           G::kCtas > 1 ? G::kCtas : 0);
    return cudaLaunchKernelEx(&cfg, fn, tm, a);
}

template <typename G, bool kSplit>
static cudaError_t grouped_tile(const GgMaps &tm, const GgArgs &a, const GroupedArgs &g, cudaStream_t stream) {
    switch (g.mode) {
        case Grouped::kGated: return grouped_as<Grouped::kGated, false, G, kSplit>(tm, a, stream);
        case Grouped::kGatedGrad: return grouped_as<Grouped::kGatedGrad, true, G, kSplit>(tm, a, stream);
        default:
            return g.transposed ? grouped_as<Grouped::kPlain, true, G, kSplit>(tm, a, stream)
                                : grouped_as<Grouped::kPlain, false, G, kSplit>(tm, a, stream);
    }
}

// Bytes of a store that rows at p with this pitch allow: 2 for 32, 1 for 16, 0 for an element.
static int store_width(const void *p, int64_t pitch_bytes) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(p) | (uint64_t)pitch_bytes;
    return bits % 32 == 0 ? 2 : (bits % 16 == 0 ? 1 : 0);
}

cudaError_t launch_grouped(const GroupedArgs &g, cudaStream_t stream) {
    GgArgs a{};
    const bool weights = g.mode == Grouped::kWeights, grad = g.mode == Grouped::kGatedGrad;
    // Small tile up to 128 rows, whatever their experts, and below 8 rows an expert up to 1024 rows.  Large /
    // small, us, gate and up with codes, down, down transposed, H = 2048, I = 768 (H = 1056, I = 352):
    //   128 rows, 4 experts of 4            12.0/10.0  7.6/7.1   11.2/8.9   (8.6/7.0   6.1/5.0   7.7/6.3)
    //   128 rows, one expert                13.7/9.3   8.5/6.1   12.1/8.1   (9.9/7.0   7.0/5.1   8.9/6.3)
    //   256 rows, 4 experts of 4            12.7/14.1  8.2/8.7   11.6/9.3   (8.9/7.3   6.4/5.2   7.9/6.3)
    //   512 rows, routed to 24              27.2/28.9  13.1/14.3 12.3/13.8  (9.0/10.5  7.9/7.6   8.2/6.9)
    //   512 rows, routed to 128: 103        96.1/94.5  50.7/48.4 53.9/49.4  (28.7/26.0 16.2/13.9 15.7/13.8)
    //   1016 rows, routed to 128: 115       105/110    55.5/52.8 58.1/53.0  (31.1/26.4 18.0/15.4 18.6/13.9)
    //   2048 rows, routed to 128: 121       111/120    57.6/63.8 62.4/63.0
    // The groups' sizes are not known here.  Rows that all go to one expert of many, whose weights every 16 of
    // them read again from L2, cost the small tile 31 us for 19 with 1016 rows and 96 for 26 with 4096: hence
    // the bound of 1024.
    const bool small = !weights && (g.rows <= 128 || (g.rows < 8 * (int64_t)g.E && g.rows < 1024));
    const uint32_t depth = small ? GgSmall::kK : GgLarge::kK;
    const uint32_t side = small ? GgSmall::kSide : GgLarge::kSide, fmt = g.half ? 0u : 1u;
    const bool a_major = !(g.transposed || grad);  // the M side's operand is channel-major
    const int elem = g.out_dtype == MOE_DT_F32 ? 4 : 2;
    a.offsets = g.offsets, a.rows = g.rows, a.E = g.E, a.C = g.channels, a.K = g.K, a.N = g.N, a.parts = g.parts;
    a.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_major ? 1u : 0u) << 15) | ((weights ? 1u : 0u) << 16) |
              ((small ? 128u : 256u) >> 4 << 24);
    a.half = elem == 2 && (g.mode == Grouped::kPlain || weights) ? g.out_dtype == MOE_DT_F16 : g.half;
    a.out32 = (g.mode == Grouped::kPlain || weights) && elem == 4;
    a.out = static_cast<unsigned char *>(g.out), a.ldo = g.ldo;
    a.vec = store_width(g.out, g.ldo * (a.out32 ? 4 : 2));
    a.p = static_cast<unsigned char *>(g.p), a.pvec = store_width(g.p, 2 * (int64_t)g.channels);
    a.code = g.code, a.codes = g.codes, a.scales = g.scales, a.pitch = microscale_pitch(2 * g.channels);
    a.status = g.status;
    a.chain = a.out32 || (g.mode == Grouped::kGated && g.codes && g.half) ? kGgChainFine : kGgChain;
    const bool split = !weights && (int64_t)g.parts * g.K > a.chain;
    a.pieces = split ? g.parts * ((g.K + a.chain - 1) / a.chain) : 1;

    GgMaps tm;
    memset(&tm, 0, sizeof tm);
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    bool ok = true;
    auto rows_map = [&](CUtensorMap *m, const void *p, int64_t cols, int64_t ld, uint32_t box) {
        const uint64_t d[2] = {(uint64_t)cols * 2, (uint64_t)g.rows}, s[1] = {(uint64_t)ld * 2};
        const uint32_t b[2] = {128, box};
        ok = ok && make_tmap_bytes(m, p, 2, d, s, b, sw);
    };
    // channels in chunks of 64, two a box
    auto deep_map = [&](CUtensorMap *m, const void *p, int64_t cols, int64_t ld) {
        const uint64_t d[3] = {128, (uint64_t)g.rows, (uint64_t)cols / 64}, s[2] = {(uint64_t)ld * 2, 128};
        const uint32_t b[3] = {128, depth, 2};
        ok = ok && make_tmap_bytes(m, p, 3, d, s, b, sw);
    };
    a.deep_m = a_major && g.mode != Grouped::kGated && g.channels % 64 == 0;
    a.deep_n = weights && g.N % 64 == 0;
    auto weights_map = [&](CUtensorMap *m, const void *p) {
        if (a.deep_m) {
            const uint64_t row = (uint64_t)g.channels * 2;
            const uint64_t d[4] = {128, (uint64_t)g.K, (uint64_t)g.channels / 64, (uint64_t)g.E}, s[3] = {row, 128, row * g.K};
            const uint32_t b[4] = {128, depth, 2, 1};
            ok = ok && make_tmap_bytes(m, p, 4, d, s, b, sw);
            return;
        }
        const uint64_t in = a_major ? g.channels : g.K, out = a_major ? g.K : g.channels;
        const uint64_t d[3] = {in * 2, out, (uint64_t)g.E}, s[2] = {in * 2, in * out * 2};
        const uint32_t b[3] = {128, a_major ? depth : 128u, 1};
        ok = ok && make_tmap_bytes(m, p, 3, d, s, b, sw);
    };
    if (weights) {
        rows_map(&tm.x, g.x, g.channels, g.ldx, depth);
        rows_map(&tm.w, g.w, g.N, g.ldw, depth);
        if (a.deep_m) deep_map(&tm.xs, g.x, g.channels, g.ldx);
        if (a.deep_n) deep_map(&tm.x2s, g.w, g.N, g.ldw);
        const uint64_t in = (uint64_t)g.N * elem;
        const uint64_t d[3] = {in, (uint64_t)g.channels, (uint64_t)g.E}, s[2] = {in, in * g.channels};
        const uint32_t b[3] = {64, 32, 1};
        ok = ok && make_tmap_bytes(&tm.y, g.out, 3, d, s, b, CU_TENSOR_MAP_SWIZZLE_64B);
    } else {
        rows_map(&tm.x, g.x, g.K, g.ldx, side);
        weights_map(&tm.w, g.w);
        if (!small) rows_map(&tm.xs, g.x, g.K, g.ldx, GgLarge::kPiece);
        if (g.parts == 2) rows_map(&tm.x2, g.x2, g.K, g.ldx, side);
        if (g.parts == 2 && !small) rows_map(&tm.x2s, g.x2, g.K, g.ldx, GgLarge::kPiece);
        if (g.w2) weights_map(&tm.w2, g.w2);
        // results: boxes of 16 rows of 32 channels, where the rows allow tensor stores and their bytes
        // fit the coordinates
        auto result_map = [&](CUtensorMap *m, void *p, int64_t cols, int64_t ld, int bytes) {
            const uint64_t d[2] = {(uint64_t)cols * bytes, (uint64_t)g.rows}, s[1] = {(uint64_t)ld * bytes};
            const uint32_t b[2] = {32u * bytes, 16};
            ok = ok && make_tmap_bytes(m, p, 2, d, s, b, bytes == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
        };
        a.bulk = g.mode == Grouped::kPlain && a.vec > 0 && a.ldo < ((int64_t)1 << 34);
        if (a.bulk) result_map(&tm.y, g.out, g.channels, g.ldo, elem);
        if (grad) result_map(&tm.y, g.out, 2 * (int64_t)g.channels, g.ldo, 2);
        if (grad && g.p) result_map(&tm.p, g.p, g.channels, g.channels, 2);
    }
    if (!ok) return cudaErrorInvalidValue;
    if (weights)
        return a.out32 ? grouped_as<Grouped::kWeights32, false, GgLarge>(tm, a, stream)
                       : grouped_as<Grouped::kWeights, false, GgLarge>(tm, a, stream);
    if (split) return small ? grouped_tile<GgSmall, true>(tm, a, g, stream) : grouped_tile<GgLarge, true>(tm, a, g, stream);
    return small ? grouped_tile<GgSmall, false>(tm, a, g, stream) : grouped_tile<GgLarge, false>(tm, a, g, stream);
}

}  // namespace moe
