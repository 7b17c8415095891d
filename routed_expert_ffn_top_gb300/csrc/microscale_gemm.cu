// microscale_gemm.cu -- the grouped product of 4-bit block-scaled rows and expert weights on
// the block-scaled tensor-core MMAs (tcgen05.mma kind::mxf4, E2M1 codes, one E8M0 scale per
// 32 along K).
//
// Rows [rows][K] are grouped by expert (offsets, as the token plan gives them); expert e's
// weights are [N][K], so
//   y[r][n] = sum_b 2^(X_r,b + X_n,b) sum_{i in block b} c_r,i c_n,i,      r in e's rows.
// Products and scales are exact; the sums over K run in the tensor core's fp32 accumulators in
// K order, so a row's result does not depend on its group, its tile or the grid.
//
// A unit is a tile of rows of one expert times a tile of its output channels (MxTile gives the
// two shapes).  Groups need no padding: a tile's row box may run into the next expert's rows,
// whose results are dropped by the epilogue (a row only reaches its own results).  The gated
// form takes a run of gate channels and the up channels beside them, computes p = SiLU(g) u in
// fp32 and quantises it in the epilogue, so g and u never leave the chip.
//
// Per CTA (persistent, one an SM), 16 warps: 0-3 and 12-15 drain the accumulators in turn, 4-7
// bring the scales through shared memory into tensor memory, 8 and 10 issue the copies of codes,
// 9 the MMAs, 11 is idle (a warp reads the tensor-memory lanes of its number modulo 4).  A stage
// is 512 of K: two chunks of 256 as 128-byte rows of codes, 128-byte swizzled.  The MMA reads
// the scale of row r at lane r % 32, column r / 32, four K blocks a 32-bit column, repeated in
// the four lane quadrants.  Accumulators are double-buffered, so a tile's epilogue overlaps the
// next one's MMAs.
//
// What bounds it, on a GB300 (H = 2048, I = 768, 128 experts, top 8 unless said):
//   few rows     HBM.  21 tokens (75 experts reached): gated 21.8 us for 126 MB (0.85 of the copy
//                rate), down 15.3 us for 63 MB (0.61: 4 us of a launch are not copies, and a unit
//                has only 48 KB).  One token: 6.8 and 5.6 us, start-up and one pass of latency.
//                In an expert step both begin while the kernel ahead runs (MxArgs::early).
//   many rows    16384 x 8192 x 8192 in one group takes 379 us (5.8 PFLOP/s, 3.0 of the bf16 rate),
//                the same with the copies of codes alone 364 (40 KB per 256 of K, which its MMAs
//                take 384 cycles for): this form is bound by its copies.
//                8192 tokens: gated 105 us (3.9 PFLOP/s; 512 rows an expert, four row tiles),
//                down 85 us, of which 16 go with the stores of y (268 MB) not issued and 7 more
//                with their staging.
// Two CTAs a tile (cta_group::2, 256 x 192) take 28 KB in for these 40, but gated 113 us, down 93, and
// the large product 374, so something other than the copies bound them, which was not found: left
// out.  So were, for few rows, both products of an expert step in
// one grid, the second waiting for the first row tile by row tile (8 tokens 44 against 38 us, 21
// the same); 256-deep stages (21 tokens' gated product 26.6 against 22.1); an L2 promotion of 256
// bytes (down 21.0 against 19.1).  Stores of y by 128-byte rows take the time of the 64-byte ones.
#include <type_traits>

#include "gemm_core.cuh"
#include "microscale.cuh"
#include "row_io.cuh"

namespace moe {

constexpr int kMxThreads = 512;
constexpr int kMxMaxSlots = 8;
constexpr int kMxScaleK = 1024;  // K per copy of scales: 32-byte rows
constexpr int kMxStaging = 2048;  // bytes a warp stages for its stores: 32 rows of 64

// Two tiles.
//   kTok = 128: 128 rows of x as the MMA's M side, 192 channels as its N side (two accumulators
//     of 192 columns leave 128 columns of tensor memory, 96 of them for the scales of two stages;
//     256 would leave none).
//   kTok = 32, for small groups: the sides change places, 128 channels are M and up to 32 rows
//     N, so no MMA reads rows that do not exist and four epilogue warps share every row (with
//     the rows on the M side one token's gated product took 8.4 us, this way 7.2).
template <int kTok_>
struct MxTile {
    static_assert(kTok_ == 32 || kTok_ == 128, "row tiles");
    static constexpr bool kSwap = kTok_ == 32;
    static constexpr int kTok = kTok_, kCh = kSwap ? 128 : 192;
    static constexpr int kA = kSwap ? kCh : kTok, kB = kSwap ? kTok : kCh;  // M and N sides
    static_assert(kA == 128, "the MMA's M");
    static constexpr int kChunks = 2;                      // 256-wide chunks of K per stage
    // Copies per stage, each behind barriers of its own: the scales and the MMA issuer go by 512
    // of K (at 256, beside the gated epilogue's instructions, they fell behind: 132 us for 118),
    // the large tile's memory is refilled by 256.
    static constexpr int kSub = kSwap ? 1 : 2;
    static constexpr int kPer = kChunks / kSub;            // chunks per copy
    static constexpr int kStageK = 256 * kChunks;
    static constexpr int kAChunk = kA * 128;               // one chunk of the M side
    static constexpr int kBChunk = kB * 128;
    static constexpr int kABytes = kChunks * kAChunk;
    static constexpr int kBBytes = kChunks * kBChunk;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kScaleBytes = (kA + kB) * 32;     // one copy of scales, M side then N side
    static constexpr int kScaleBufs = kSwap ? 6 : 4;
    static constexpr int kStages = kSwap ? 4 : 2;
    static constexpr int kACols = kA / 32;                 // scale columns per 128 of K
    static constexpr int kBCols = kB / 32;
    static constexpr int kBPad = (kBCols + 3) / 4 * 4;     // every set starts at a multiple of 4
    static constexpr int kGroups = 2 * kChunks;            // 128-wide groups of K per stage
    static_assert(kGroups == 4, "a stage's scales of a row are one 16-byte piece");
    static constexpr int kSfCols = kGroups * (kACols + kBPad);  // per stage
    static constexpr int kSfCol0 = 2 * kB;                 // after the two accumulators
    static constexpr uint32_t kTmemCols = kSfCol0 + kStages * kSfCols <= 256 ? 256 : 512;
    static constexpr size_t kSmem = (size_t)kStages * kStageBytes + kScaleBufs * kScaleBytes + 1024 +
                                    (kSwap ? 0 : 8 * kMxStaging);
    static_assert(kStageBytes % 1024 == 0 && kScaleBytes % 512 == 0, "stage alignment");
    static_assert(kSfCol0 + kStages * kSfCols <= 512, "tensor memory");
    static constexpr int kSlots = kStages * kSub;
    static_assert(kSlots <= kMxMaxSlots, "barriers");
};

struct MxCtl {
    uint64_t full[kMxMaxSlots];        // per copy slot
    uint64_t empty[kMxMaxSlots];
    uint64_t sfull[kMxMaxSlots];      // the stage's scales are in tensor memory
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t done;
    uint32_t tmem;
    volatile int abort;
    int32_t wsum[kMxThreads / 32];
    int32_t valid_rows;
    int32_t first[kMicroscaleMaxExperts + 1];  // row tiles before expert e
    int32_t begin[kMicroscaleMaxExperts + 1];  // first row of expert e
};

// gwait with the first tries made without reading the timer, whose latency would add to
// every wait that is short.
__device__ __forceinline__ bool mx_wait(uint64_t *bar, uint32_t parity, MxCtl &ctl) {
    for (int i = 0; i < 32; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return gwait(bar, parity, ctl);
}

// The same for a whole warp, with one answer.
__device__ __forceinline__ bool mx_warp_wait(uint64_t *bar, uint32_t parity, MxCtl &ctl) {
    return __all_sync(0xffffffffu, mx_wait(bar, parity, ctl));
}

struct MxArgs {
    // early: offsets, ids and weights were complete before the kernel ahead began.  ids: the
    // groups' sizes are counted from nids <= kMxThreads routes' experts instead.
    int early, nids;
    const int32_t *ids;
    int deep;                // the maps' third dimension is K's 256-wide chunks, a stage a copy
    const int32_t *offsets;  // NULL: one group of all rows
    const uint8_t *x_scales, *w_scales;
    int kpitch;              // their row bytes
    int64_t rows;
    int E, N, K;
    int nct;                 // column tiles
    int dt, dct;             // a step of a CTA's units in row tiles and column tiles
    int vec, bulk;           // y rows allow 32-byte stores, tensor stores
    void *y;
    int64_t ldy;
    uint8_t *codes, *scales;  // gated output
    int pitch;                // its scale row bytes
    int32_t *status;
};

// Instruction descriptor of kind::mxf4 with M = 128: E2M1 A and B (K-major), E8M0 scales; the
// scale ids pick the 16-bit half of the scale columns (0: bytes 0-1, 2: bytes 2-3).
__device__ __forceinline__ constexpr uint32_t mx_idesc(int N, uint32_t sf_id) {
    return (sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
           ((uint32_t)(128 >> 4) << 24) | (sf_id << 29);
}

__device__ __forceinline__ void umma_mxf4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// 32 columns of one row from column n: whole 32-byte sectors where the row allows.
template <typename T>
__device__ __forceinline__ void store_row32(const MxArgs &a, int64_t row, int n, const uint32_t (&v)[32]) {
    T *dst = static_cast<T *>(a.y) + row * a.ldy + n;
    if (a.vec && n + 32 <= a.N) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) st_global_32(dst + i, &v[i]);
        } else {
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = pack2<T>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            st_global_32(dst, &o[0]);
            st_global_32(dst + 16, &o[8]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (n + i < a.N) put_f32(dst + i, __uint_as_float(v[i]));
}

// SiLU(g) u = g u / (1 + 2^(-g log2 e)) by the approximate power and reciprocal: within 2^-21
// (1 + |g| / 4) of its value for negative g, 2^-21 for others, and p goes to 4 bits next.  Below
// g = -87.3 the reciprocal is 0, and so is the result, whose value is under 2^-119 |u|.  (expf and the division took the gated epilogue's
// instructions from 8 to 16 a value.)
__device__ __forceinline__ float gate(float g, float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return g * r * u;
}

// A CTA's units: u = blockIdx.x, blockIdx.x + gridDim.x, ...; unit u is channel tile u % nct of
// row tile u / nct.  Each warp walks them on its own, without dividing, and finds the next
// expert with its 32 lanes at once: a walk by one thread took 1000 cycles a unit, as long as a
// small unit's copies.
template <int kM>
struct MxWalk {
    int t, ct, e;          // row tile, channel tile, expert
    int dt, dct;           // a step
    int nrows;             // of this row tile
    int row0;

    __device__ __forceinline__ void place(const MxArgs &a, const MxCtl &ctl) {
        unsigned past;
        do {
            const int i = e + 1 + (threadIdx.x & 31);
            past = __ballot_sync(0xffffffffu, i <= a.E && ctl.first[i] <= t);
            e += __popc(past);
        } while (past == 0xffffffffu);
        row0 = ctl.begin[e] + (t - ctl.first[e]) * kM;
        const int left = ctl.begin[e + 1] - row0;
        nrows = left < kM ? left : kM;
    }
    __device__ __forceinline__ MxWalk(const MxArgs &a, const MxCtl &ctl, int tiles) {
        t = blockIdx.x / a.nct, ct = blockIdx.x % a.nct, e = 0;
        dt = a.dt, dct = a.dct;
        if (t < tiles) place(a, ctl);
    }
    __device__ __forceinline__ void next(const MxArgs &a, const MxCtl &ctl, int tiles) {
        t += dt, ct += dct;
        if (ct >= a.nct) ct -= a.nct, ++t;
        if (t < tiles) place(a, ctl);
    }
};

// The 16 scale bytes (512 of K) number `piece` of a row of a copy.  Rows are 32 bytes, their two
// pieces exchanged in every other four rows, so that 8 lanes reading a piece each take all banks.
__device__ __forceinline__ int mx_scale_at(int row, int piece) { return row * 32 + ((piece ^ ((row >> 2) & 1)) << 4); }
__device__ __forceinline__ uint4 mx_scale_piece(const unsigned char *base, int row, int piece) {
    return *reinterpret_cast<const uint4 *>(base + mx_scale_at(row, piece));
}

// The four words of a stage's piece to w[0], w[kStep], ...
template <int kStep>
__device__ __forceinline__ void mx_scale_words(const uint4 &v, const uint32_t (&mask)[4], uint32_t *w) {
    w[0] = v.x & mask[0];
    w[kStep] = v.y & mask[1];
    w[2 * kStep] = v.z & mask[2];
    w[3 * kStep] = v.w & mask[3];
}

// 32 rows x 32 columns of a warp by tensor stores of 64-byte rows through its staging memory (a
// lane's own 32 bytes of a row at a time, 32 rows an instruction, took up to a third of a
// product's time).  byte0: of the first column in its row.
template <typename T>
__device__ __forceinline__ void mx_store_bulk(const CUtensorMap &tm_y, unsigned char *staging, int byte0, int row0,
                                              int lane, const uint32_t (&v)[32]) {
    constexpr int kParts = sizeof(T) / 2;  // 64-byte rows: 32 columns of 16 bits, 16 of 32
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
        if (lane == 0) bulk_store_wait<true>();  // the staging memory's last store has been read
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 o;
            if constexpr (sizeof(T) == 4) {
                o = make_uint4(v[16 * q + 4 * i], v[16 * q + 4 * i + 1], v[16 * q + 4 * i + 2], v[16 * q + 4 * i + 3]);
            } else {
                uint32_t w[4];
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    w[p] = pack2<T>(__uint_as_float(v[8 * i + 2 * p]), __uint_as_float(v[8 * i + 2 * p + 1]));
                o = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<uint4 *>(staging + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) = o;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            asm volatile(
                "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\t"
                "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(&tm_y)),
                "r"(byte0 + 64 * q), "r"(row0), "r"(smem_u32(staging))
                : "memory");
    }
}

// Small tile: lane's channel n of up to 32 rows (v: one per row).
template <typename T>
__device__ __forceinline__ void mx_store_columns(const MxArgs &a, int row0, int nrows, int n, const uint32_t (&v)[32]) {
    if (n >= a.N) return;
    T *dst = static_cast<T *>(a.y) + (int64_t)row0 * a.ldy + n;
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j < nrows) put_f32(dst + j * a.ldy, __uint_as_float(v[j]));
}

// Small gated tile: warps 0 and 1 hold g of 64 channels, warps 2 and 3 u of the same; u goes
// through shared memory, a block of 32 channels is a warp's lanes.
__device__ __forceinline__ void mx_gate_columns(const MxArgs &a, float *exchange, int group, int row0, int nrows, int n0, int warp,
                                                int lane, const uint32_t (&v)[32], bool last) {
    float *u = exchange + (32 * warp + lane) % 64;
    if (warp >= 2) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < nrows) u[64 * j] = __uint_as_float(v[j]);
    }
    named_bar_sync(1 + 2 * group, 128);
    const int I = a.N / 2, n = n0 + 32 * warp;
    if (warp < 2 && n < I) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j >= nrows) break;
            const float p = gate(__uint_as_float(v[j]), u[64 * j]);
            const uint32_t byte = microscale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(p) & 0x7fffffffu));
            uint32_t c = byte == 255u ? 0u : fp4(p * microscale_inverse(byte)) << (4 * (lane & 7));
            c |= __shfl_xor_sync(0xffffffffu, c, 1);
            c |= __shfl_xor_sync(0xffffffffu, c, 2);
            c |= __shfl_xor_sync(0xffffffffu, c, 4);
            const int64_t row = row0 + j;
            if ((lane & 7) == 0) *reinterpret_cast<uint32_t *>(a.codes + row * (I / 2) + n / 2 + lane / 2) = c;
            if (lane == 0) a.scales[row * a.pitch + n / 32] = (uint8_t)byte;
        }
    }
    if (warp == 2 && last)
        for (int j = 0; j < nrows; ++j)
            for (int b = I / 32 + lane; b < a.pitch; b += 32) a.scales[(int64_t)(row0 + j) * a.pitch + b] = 0;
    named_bar_sync(1 + 2 * group, 128);  // u may be written over
}

// First weight row of a unit: of the tile's channels, or (gated) of its gate channels, whose up
// rows lie N / 2 further on.
template <bool kGated, int kCh>
__device__ __forceinline__ int mx_first_channel(const MxArgs &a, int e, int ct) {
    return e * a.N + ct * (kGated ? kCh / 2 : kCh);
}

// kOut: 0 bf16, 1 f16, 2 f32, 3 gated codes and scales.
template <int kTok, int kOut>
__global__ void __launch_bounds__(kMxThreads, 1)
microscale_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ CUtensorMap tm_y, const MxArgs a) {
    using G = MxTile<kTok>;
    constexpr bool kGated = kOut == 3;
    constexpr int kN = G::kB, kHalf = G::kCh / 2;
    using Out = typename std::conditional<kOut == 0, __nv_bfloat16,
                                          typename std::conditional<kOut == 1, __half, float>::type>::type;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *stages = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *scales = stages + G::kStages * G::kStageBytes;
    __shared__ MxCtl ctl;
    __shared__ float exchange[kGated && G::kSwap ? 2 * 32 * 64 : 1];  // u of the gated small tile, one unit a group
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kSlots; ++s) {
            mbar_init(&ctl.full[s], 2);  // the two code producers
            mbar_init(&ctl.empty[s], 1);
        }
        for (int s = 0; s < G::kStages; ++s) mbar_init(&ctl.sfull[s], 4);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl.tfull[b], 1);
            mbar_init(&ctl.tempty[b], 4);
        }
        mbar_init(&ctl.done, 1);
        ctl.abort = 0;
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(&ctl.tmem, G::kTmemCols);
    if (warp == 8 && lane == 0) {
        prefetch_tensormap(&tm_w);
        prefetch_tensormap(&tm_x);
    }
    // Early, nothing of the kernel ahead is needed before the rows: the tiles are counted and the
    // first weights copied while it runs.
    if (!a.early) {
        pdl_wait();
        pdl_launch_dependents();
    }
    if (a.ids) {
        for (int e = threadIdx.x; e < a.E; e += kMxThreads) ctl.begin[e] = 0;
        __syncthreads();
        const int id = (int)threadIdx.x < a.nids ? __ldcg(a.ids + threadIdx.x) : -1;
        if (id >= 0 && id < a.E) atomicAdd(&ctl.begin[id], 1);
        __syncthreads();
    }

    // row tiles before each expert; offsets outside [0, rows] or running backwards are clamped.
    // Counted groups' rows are summed along, in the upper half of the same words.
    const int low = a.ids ? 0xffff : -1;
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += kMxThreads) {
        const int e = e0 + threadIdx.x;
        int64_t lo = 0, hi = 0;
        if (e < a.E) {
            if (a.ids) {
                hi = ctl.begin[e];
            } else {
                if (!a.offsets) hi = a.rows;
                else if (a.early) lo = __ldcg(a.offsets + e), hi = __ldcg(a.offsets + e + 1);
                else lo = a.offsets[e], hi = a.offsets[e + 1];
                lo = lo < 0 ? 0 : (lo > a.rows ? a.rows : lo);
                hi = hi < lo ? lo : (hi > a.rows ? a.rows : hi);
            }
        }
        const int tiles = (int)((hi - lo + kTok - 1) / kTok) | (a.ids ? (int)hi << 16 : 0);
        int inc = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += t;
        }
        if (lane == 31) ctl.wsum[warp] = inc;
        __syncthreads();
        int off = carry, chunk = 0;
        for (int w = 0; w < kMxThreads / 32; ++w) {
            const int t = ctl.wsum[w];
            if (w < warp) off += t;
            chunk += t;
        }
        if (e < a.E) {
            const int end = off + inc, at = end - tiles;
            ctl.first[e] = at & low;
            ctl.begin[e] = a.ids ? at >> 16 : (int)lo;
            if (e == a.E - 1) {
                ctl.first[a.E] = end & low;
                ctl.valid_rows = ctl.begin[a.E] = a.ids ? end >> 16 : (int)hi;
            }
        }
        carry += chunk;
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (Warp 8 reads weights only.)  Either way the next kernel may begin only after this one's
    // wait: its beginning says that the kernel ahead of this one is complete.
    if (a.early && warp != 8) {
        pdl_wait();
        pdl_launch_dependents();
    }
    const int tiles = carry & low;
    const int nks = (a.K + G::kStageK - 1) / G::kStageK;  // stages per unit
    constexpr int kPerScale = kMxScaleK / G::kStageK;         // stages per copy of scales

    if (warp == 8 || warp == 10) {
        // two producer warps: weight codes and row codes
        // weights that one row tile reads leave L2 first, rows (read by every channel tile) last:
        // with layers' weights in turn, 21 tokens' gated product 23.2 to 21.5 us, 256 tokens' down
        // product 23.2 to 20.0
        const uint64_t keep = warp == 8 ? policy_evict_normal() : policy_evict_last();
        const uint64_t once = warp == 8 ? policy_evict_first() : keep;
        const bool side_a = G::kSwap == (warp == 8);
        const int chunk = side_a ? G::kAChunk : G::kBChunk;
        unsigned char *const base = stages + (side_a ? 0 : G::kABytes);
        int stage = 0;
        uint32_t phase = 0, issued = 0, par = 0;
        bool ok = true, ahead = a.early && warp == 8;
        for (MxWalk<kTok> x(a, ctl, tiles); x.t < tiles && ok; x.next(a, ctl, tiles)) {
            const int w0 = mx_first_channel<kGated, G::kCh>(a, x.e, x.ct);
            const uint64_t pol = ctl.first[x.e + 1] - ctl.first[x.e] == 1 ? once : keep;
            for (int s = 0; s < nks && ok; ++s) {
#pragma unroll
                for (int b = 0; b < G::kSub; ++b) {
                    const int slot = stage * G::kSub + b;
                    if (!(ok = mx_warp_wait(&ctl.empty[slot], phase ^ 1u, ctl))) break;
                    if (lane == 0) {
                        // one copy brings the slot's chunks, or one a chunk (past K: none)
                        uint64_t *bar = &ctl.full[slot];
                        const int c0 = s * G::kChunks + b * G::kPer, left = (a.K + 255) / 256 - c0;
                        const int copies = left <= 0 ? 0 : a.deep ? 1 : (left < G::kPer ? left : G::kPer);
                        unsigned char *dst = base + stage * G::kStageBytes + b * G::kPer * chunk;
                        mbar_arrive_expect_tx(bar, (a.deep && copies ? G::kPer : copies) * chunk);
                        for (int c = 0; c < copies; ++c, dst += chunk) {
                            const int cx = a.deep ? 0 : (c0 + c) * 128, cz = a.deep ? c0 : 0;
                            if (warp == 8) tma_load_4d(dst, &tm_w, cx, w0, 0, cz, bar, pol);
                            else tma_load_3d(dst, &tm_x, cx, x.row0, cz, bar, pol);
                        }
                    }
                    __syncwarp();
                    issued |= 1u << slot;
                    par = (par & ~(1u << slot)) | (phase << slot);
                }
                if (++stage == G::kStages) {
                    stage = 0, phase ^= 1u;
                    // all slots full: the kernel ahead is waited for outside the bounded waits
                    if (ahead) pdl_wait(), ahead = false;
                }
            }
        }
        // fewer stages than the ring holds: the other producer's copies come after the kernel ahead
        if (ahead) pdl_wait();
        // every copy has landed before the CTA can exit
        for (int s = 0; s < G::kSlots; ++s)
            if ((issued >> s) & 1u)
                if (!mbar_wait_bounded(&ctl.full[s], (par >> s) & 1u)) ctl.abort = 1;
        __syncwarp();
    } else if (warp == 9) {
        if (lane == 0) {
            // K-major, 128-byte swizzle: 32 bytes per K step, 8-row atoms 1 KB apart.  A step
            // only moves the address field of the descriptors (16-byte units).
            const uint64_t a0 = umma_smem_desc(smem_u32(stages), 16, 1024, 2);
            const uint64_t b0 = umma_smem_desc(smem_u32(stages) + G::kABytes, 16, 1024, 2);
            int stage = 0, buf = 0;
            uint32_t phase = 0, tphase = 1;
            const int dt = a.dt, dct = a.dct;
            for (int t = blockIdx.x / a.nct, ct = blockIdx.x % a.nct; t < tiles && !ctl.abort;) {
                if (!mx_wait(&ctl.tempty[buf], tphase, ctl)) break;
                const uint32_t d = ctl.tmem + (uint32_t)(buf * kN);
                bool ok = true;
                for (int s = 0; s < nks && ok; ++s) {
                    const uint64_t ad = a0 + (uint32_t)(stage * (G::kStageBytes >> 4));
                    const uint64_t bd = b0 + (uint32_t)(stage * (G::kStageBytes >> 4));
                    const uint32_t sf = ctl.tmem + (uint32_t)(G::kSfCol0 + stage * G::kSfCols);
                    const int left = (a.K - s * G::kStageK + 63) / 64;  // K steps of this stage
                    auto step = [&](int ks) {
                        umma_mxf4(d, ad + (ks >> 2) * (G::kAChunk >> 4) + (ks & 3) * 2,
                                  bd + (ks >> 2) * (G::kBChunk >> 4) + (ks & 3) * 2, mx_idesc(kN, (ks & 1) ? 2u : 0u),
                                  sf + (ks >> 1) * G::kACols, sf + G::kGroups * G::kACols + (ks >> 1) * G::kBPad,
                                  s > 0 || ks > 0);
                    };
#pragma unroll
                    for (int b = 0; b < G::kSub; ++b) {
                        const int slot = stage * G::kSub + b;
                        constexpr int kSteps = G::kPer * 4;  // K steps a slot
                        if (!(ok = mx_wait(&ctl.full[slot], phase, ctl) && (b > 0 || mx_wait(&ctl.sfull[stage], phase, ctl))))
                            break;
                        tc_fence_after();
                        if (left >= (b + 1) * kSteps) {
#pragma unroll
                            for (int ks = 0; ks < kSteps; ++ks) step(b * kSteps + ks);
                        } else {
                            for (int ks = b * kSteps; ks < left; ++ks) step(ks);
                        }
                        umma_commit(&ctl.empty[slot]);
                    }
                    if (++stage == G::kStages) stage = 0, phase ^= 1u;
                }
                if (!ok) break;
                umma_commit(&ctl.tfull[buf]);
                if (buf) tphase ^= 1u;
                buf ^= 1;
                t += dt, ct += dct;
                if (ct >= a.nct) ct -= a.nct, ++t;
            }
            // every issued MMA has completed before the CTA frees its tensor memory
            umma_commit(&ctl.done);
            if (!mbar_wait_bounded(&ctl.done, 0)) ctl.abort = 1;
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // scales: copied kMxScaleK of K at a time, kScaleBufs copies ahead, by 16-byte cp.async
        // (a tensor copy of 64-byte rows takes 11 cycles a row, as long as the unit's codes
        // when K is short); every warp then needs all rows, hence the barrier
        const uint32_t quad = (uint32_t)(32 * (warp - 4)) << 16;
        const int nb = a.K / 32, per_unit = (nks + kPerScale - 1) / kPerScale;
        MxWalk<kTok> ahead(a, ctl, tiles);
        int part_a = 0, slot_a = 0, slot = 0, stage = 0;
        uint32_t phase = 0;
        auto issue = [&]() {
            if (ahead.t < tiles) {
                const int w0 = mx_first_channel<kGated, G::kCh>(a, ahead.e, ahead.ct);
                unsigned char *S = scales + slot_a * G::kScaleBytes;
#pragma unroll
                for (int i = 0; i < ((G::kA + G::kB) * 2 + 127) / 128; ++i) {
                    const int p = (int)threadIdx.x - 128 + 128 * i, r = p >> 1, c = p & 1;
                    const int rs = r < G::kA ? r : r - G::kA;  // row of its side
                    const bool is_w = (r < G::kA) == G::kSwap;
                    int64_t row = is_w ? w0 + rs : ahead.row0 + rs;
                    if (kGated && is_w && rs >= kHalf) row += a.N / 2 - kHalf;
                    const bool in = r < G::kA + G::kB && row < (is_w ? (int64_t)a.E * a.N : a.rows) &&
                                    part_a * 32 + c * 16 < a.kpitch;
                    if (in)
                        cp_async_16(S + mx_scale_at(r, c),
                                    (is_w ? a.w_scales : a.x_scales) + row * a.kpitch + part_a * 32 + c * 16);
                }
                if (++part_a == per_unit) part_a = 0, ahead.next(a, ctl, tiles);
            }
            cp_async_commit();
            if (++slot_a == G::kScaleBufs) slot_a = 0;
        };
        for (int i = 0; i < G::kScaleBufs - 1; ++i) issue();
        // after a wait that gave up the loop runs on without waits, so that the barriers stay paired
        bool ok = true;
        for (int64_t u = blockIdx.x; u < (int64_t)tiles * a.nct; u += gridDim.x)
            for (int s = 0; s < nks; ++s) {
                const int part = s % kPerScale;
                if (part == 0) {
                    if (s > 0 || u != blockIdx.x) slot = slot + 1 == G::kScaleBufs ? 0 : slot + 1;
                    cp_async_wait_group<G::kScaleBufs - 2>();
                    named_bar_sync(2, 128);
                    issue();  // into the slot that every warp has just finished with
                }
                // blocks past K have zero codes; their scale must not be a NaN
                uint32_t mask[G::kGroups];
#pragma unroll
                for (int q = 0; q < G::kGroups; ++q) {
                    const int left = nb - (s * G::kGroups + q) * 4;
                    mask[q] = left >= 4 ? 0xffffffffu : (left <= 0 ? 0u : (1u << (8 * left)) - 1u);
                }
                const unsigned char *S = scales + slot * G::kScaleBytes;
                uint4 piece[G::kACols + G::kBCols];
#pragma unroll
                for (int c = 0; c < G::kACols + G::kBCols; ++c) piece[c] = mx_scale_piece(S, c * 32 + lane, part);
                uint32_t wa[G::kGroups * G::kACols] = {}, wb[G::kGroups * G::kBPad] = {};
#pragma unroll
                for (int c = 0; c < G::kACols; ++c) mx_scale_words<G::kACols>(piece[c], mask, wa + c);
#pragma unroll
                for (int c = 0; c < G::kBCols; ++c) mx_scale_words<G::kBPad>(piece[G::kACols + c], mask, wb + c);
                // the MMAs that read this slot's scales have completed
                ok = ok && mx_warp_wait(&ctl.empty[stage * G::kSub + G::kSub - 1], phase ^ 1u, ctl);
                if (ok) {
                    tc_fence_after();
                    const uint32_t sf = ctl.tmem + quad + (uint32_t)(G::kSfCol0 + stage * G::kSfCols);
#pragma unroll
                    for (int i = 0; i < G::kGroups * G::kACols; i += 8) tmem_st8(sf + i, wa + i);
#pragma unroll
                    for (int i = 0; i < G::kGroups * G::kBPad; i += 8) tmem_st8(sf + G::kGroups * G::kACols + i, wb + i);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.sfull[stage]);
                }
                if (++stage == G::kStages) stage = 0, phase ^= 1u;
            }
        cp_async_wait_all();
    } else if (warp < 4 || warp >= 12) {
        // two groups of four warps take the accumulators, and so the units, in turn
        const int group = warp >> 3, w4 = warp & 3;
        const uint32_t quad = (uint32_t)(32 * w4) << 16;
        unsigned char *const staging = scales + G::kScaleBufs * G::kScaleBytes + (4 * group + w4) * kMxStaging;
        int local = 0;
        for (MxWalk<kTok> x(a, ctl, tiles); x.t < tiles; x.next(a, ctl, tiles), ++local) {
            const int buf = local & 1;
            if (buf != group) continue;
            if (!mx_warp_wait(&ctl.tfull[buf], (uint32_t)(local >> 1) & 1u, ctl)) {
                if constexpr (!(kGated && G::kSwap)) break;
                named_bar_sync(1 + 2 * group, 128);  // a warp that does not give up waits there for the others
                named_bar_sync(1 + 2 * group, 128);
                continue;
            }
            tc_fence_after();
            const uint32_t d = ctl.tmem + quad + (uint32_t)(buf * kN);
            const int n0 = x.ct * (kGated ? kHalf : G::kCh);
            if constexpr (G::kSwap) {
                uint32_t v[32];
                tmem_ld32(d, v);
                tmem_ld_wait(v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.tempty[buf]);
                if constexpr (!kGated) mx_store_columns<Out>(a, x.row0, x.nrows, n0 + 32 * w4 + lane, v);
                else mx_gate_columns(a, exchange + group * (32 * 64), group, x.row0, x.nrows, n0, w4, lane, v, x.ct == a.nct - 1);
                continue;
            }
            const int64_t row = (int64_t)x.row0 + 32 * w4 + lane;
            const bool live = 32 * w4 + lane < x.nrows;
            if (32 * w4 >= x.nrows) {
                // no row of this warp's lanes: the accumulator holds nothing of the tile here
            } else if constexpr (!kGated) {
                const bool bulk = a.bulk && 32 * w4 + 32 <= x.nrows;
#pragma unroll 1
                for (int c = 0; c < kN && n0 + c < a.N; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(d + c, v);
                    tmem_ld_wait(v);
                    if (bulk) mx_store_bulk<Out>(tm_y, staging, (n0 + c) * (int)sizeof(Out), x.row0 + 32 * w4, lane, v);
                    else if (live) store_row32<Out>(a, row, n0 + c, v);
                }
            } else {
                const int I = a.N / 2;
#pragma unroll 1
                for (int c = 0; c < kHalf && n0 + c < I; c += 32) {
                    uint32_t g[32], up[32];
                    tmem_ld32(d + c, g);
                    tmem_ld32(d + kHalf + c, up);
                    tmem_ld_wait(g);
                    tmem_ld_wait(up);
                    float p[32], top = 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) p[i] = gate(__uint_as_float(g[i]), __uint_as_float(up[i]));
#pragma unroll
                    for (int i = 0; i < 32; i += 2) top = max_abs(top, p[i], p[i + 1]);
                    const uint32_t byte = microscale_byte(__float_as_uint(top) & 0x7fffffffu);
                    const float inv = microscale_inverse(byte);
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float f[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = p[8 * q + i] * inv;
                        o[q] = byte == 255u ? 0u : fp4x8(f);
                    }
                    if (live) {
                        *reinterpret_cast<uint4 *>(a.codes + row * (I / 2) + (n0 + c) / 2) = make_uint4(o[0], o[1], o[2], o[3]);
                        a.scales[row * a.pitch + (n0 + c) / 32] = (uint8_t)byte;
                    }
                }
                if (live && x.ct == a.nct - 1)
                    for (int b = I / 32; b < a.pitch; ++b) a.scales[row * a.pitch + b] = 0;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.tempty[buf]);
        }
        if (lane == 0) bulk_store_wait<false>();  // stores have left shared memory and are visible
        // rows past the last group (dropped routes): zeros
        for (int64_t r = ctl.valid_rows + (int64_t)blockIdx.x; r < a.rows && group == 0; r += gridDim.x) {
            if constexpr (kGated) {
                for (int i = threadIdx.x; i < a.N / 64; i += 128)
                    *reinterpret_cast<uint4 *>(a.codes + r * (a.N / 4) + 16 * i) = uint4{0, 0, 0, 0};
                for (int i = threadIdx.x; i < a.pitch; i += 128) a.scales[r * a.pitch + i] = 0;
            } else {
                for (int i = threadIdx.x; i < a.N; i += 128) put_f32(static_cast<Out *>(a.y) + r * a.ldy + i, 0.0f);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(ctl.tmem, G::kTmemCols);
    if (threadIdx.x == 0 && ctl.abort) atomicOr(a.status, MOE_DEV_WAIT_TIMEOUT);
}

// ----------------------------------------------------------------------------------- launcher
// Small tiles while the groups are small: up to 32 rows, or under 4 rows an expert on average.
// Both tiles measured over an expert step (H = 2048, I = 768, 128 experts, top 8, us, large /
// small): 1 token 17.6 / 15.8, 8 34.7 / 31.4, 21 45.4 / 44.5, 32 50.7 / 50.7, 64 (4 rows an
// expert) 55.6 / 56.4, 128 61.6 / 64.7, 256 67.1 / 75.0, 512 74.3 / 107.
MicroscaleTile microscale_tile(int64_t rows, int E) {
    using Large = MxTile<128>;
    using Small = MxTile<32>;
    return rows > 32 && rows >= 4 * (int64_t)E ? MicroscaleTile{128, Large::kCh, Large::kPer}
                                               : MicroscaleTile{32, Small::kCh, Small::kPer};
}

template <int kTok, int kOut>
static cudaError_t gemm_as(const MicroscaleMaps &tm, MxArgs a, cudaStream_t stream) {
    using G = MxTile<kTok>;
    const int per = kOut == 3 ? G::kCh / 2 : G::kCh, cols = kOut == 3 ? a.N / 2 : a.N;
    a.nct = (cols + per - 1) / per;
    const int64_t tiles = a.rows < a.E ? a.rows : a.rows / kTok + a.E;
    const int64_t units = tiles * a.nct, sms = num_sms();
    const int64_t grid = units < 1 ? 1 : (units < sms ? units : sms);
    a.dt = (int)(grid / a.nct), a.dct = (int)(grid % a.nct);
    const auto fn = microscale_gemm_kernel<kTok, kOut>;
    cudaError_t err = ensure_smem((const void *)fn, G::kSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)grid), dim3(kMxThreads), G::kSmem, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, fn, tm.x, tm.w, tm.y, a);
}

template <int kTok>
static cudaError_t gemm_tile(const MicroscaleMaps &tm, const MxArgs &a, int out, cudaStream_t stream) {
    switch (out) {
        case MOE_DT_BF16: return gemm_as<kTok, 0>(tm, a, stream);
        case MOE_DT_F16: return gemm_as<kTok, 1>(tm, a, stream);
        case MOE_DT_F32: return gemm_as<kTok, 2>(tm, a, stream);
        default: return gemm_as<kTok, 3>(tm, a, stream);
    }
}

cudaError_t launch_microscale_gemm(const MicroscaleMaps &tm, int64_t rows, const int32_t *offsets, int E,
                                   int N, int K, int dtype, void *y, int64_t ldy, uint8_t *codes,
                                   uint8_t *scales, MicroscaleEarly early, int32_t *status, cudaStream_t stream) {
    MxArgs a{};
    a.early = early.on, a.ids = early.ids, a.nids = early.nids;
    a.deep = tm.deep;
    a.offsets = offsets, a.rows = rows, a.E = E, a.N = N, a.K = K;
    a.x_scales = tm.x_scales, a.w_scales = tm.w_scales, a.kpitch = microscale_pitch(K);
    a.y = y, a.ldy = ldy, a.codes = codes, a.scales = scales, a.status = status;
    a.pitch = microscale_pitch(N / 2);
    const int elem = dtype == MOE_DT_F32 ? 4 : 2;
    a.vec = y && (reinterpret_cast<uintptr_t>(y) | (uint64_t)(ldy * elem)) % 32 == 0;
    a.bulk = tm.bulk;
    const int out = codes ? 3 : dtype;
    return microscale_tile(rows, E).m == 128 ? gemm_tile<128>(tm, a, out, stream) : gemm_tile<32>(tm, a, out, stream);
}

}  // namespace moe
