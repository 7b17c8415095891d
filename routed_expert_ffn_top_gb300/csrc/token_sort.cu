// token_sort.cu -- tokens sorted by expert and back, for prompts and for training.
//
// Routes r = m*k + j are put in (expert, r) order without padding: row i of the sorted order
// belongs to one route, expert e owns rows offsets[e] .. offsets[e+1].  A route whose expert
// id lies outside [0, E) is dropped; it still owns one row, past offsets[E], and its
// route_row entry is the bitwise complement of that row.  So every row is written by exactly
// one route and no kernel needs a row count.
//
//   plan:          route_row (a bijection of routes to rows), row_route, offsets
//   sort:          rows[row(m,j)] = x[m]                       (dropped: zeros)
//   its gradient:  gx[m] = sum_j grows[row(m,j)]
//   unsort:        out[m] = residual[m] + sum_j w[m,j] rows[row(m,j)]
//   its gradients: grows[row(m,j)] = w[m,j] gout[m]  (dropped: zeros),
//                  gw[m,j] = <gout[m], rows[row(m,j)]>         (dropped: 0)
//
// All sums are fp32 in fixed orders (slots ascending; columns by thread, then a fixed tree),
// so results are bitwise reproducible.  A value is rounded once, when it is stored.
#include <type_traits>

#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {

// ------------------------------------------------------------------------------------- plan
// Clusters of C CTAs.  Each warp of a cluster takes a contiguous run of routes and counts them
// per expert in its own row of shared memory, 32 routes a step: the lanes that share an expert
// find each other by one ballot per bit of its number, so a route's rank inside its warp's run
// needs no atomics and follows r.  Two scans (over the warps of a CTA, then over the CTAs of the
// cluster, through distributed shared memory) and one over the experts turn ranks into rows.
// Dropped routes use bucket E, which follows the last expert.
//
// What bounds it is latency, and for many routes the scattered stores of row_route, one sector a
// cycle and SM.  So several clusters count all the routes, and each writes its share of every
// warp's steps: counting again costs less than 8 SMs' stores (65,536 routes, 128 experts: 9.1 us,
// one cluster 16; 8 routes 2.0 us; 262,144 routes 26 us).  Eight clusters suffice up to there.  Past
// it a cluster still writes kPlanKeep steps of a run, whose ranks its registers hold, so clusters
// are added, all of which count all routes: 2^20 routes 0.27 ms, 2^22 3.0 ms, 2^24 47 ms, growing
// with the square.
constexpr int kPlanMaxCluster = 8;
constexpr int kPlanMaxShares = 8;  // clusters
constexpr int kPlanKeep = 4;       // steps of a share whose ranks stay in registers

struct PlanArgs {
    const int32_t *ids;
    int32_t *offsets, *row_route, *route_row;
    int R, E;
    int bits;      // of a bucket number
    int per_warp;  // routes per warp, a multiple of 32
    int nwarps;    // warps per CTA that hold routes
    int C;         // CTAs per cluster
    int share;     // steps of a warp that one cluster writes, at most kPlanKeep
};

__device__ __forceinline__ int plan_key(const PlanArgs &a, int r, int hi) {
    if (r >= hi) return -1;
    const int id = a.ids[r];
    return (uint32_t)id < (uint32_t)a.E ? id : a.E;
}

__global__ void __launch_bounds__(1024) token_plan_kernel(const PlanArgs a) {
    extern __shared__ int32_t sm[];
    const int B = a.E + 1;                       // buckets
    int32_t *cnt = sm;                           // [nwarps][B]
    int32_t *tot = cnt + a.nwarps * B;           // [C][B] every CTA's totals
    int32_t *base = tot + kPlanMaxCluster * B;   // [B]
    __shared__ int32_t wsum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int C = a.C, c = blockIdx.x % C, first_step = blockIdx.x / C * a.share;

    for (int i = threadIdx.x; i < a.nwarps * B; i += blockDim.x) cnt[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    if (C > 1) cluster_sync();  // every CTA runs before any writes another's shared memory
    else __syncthreads();

    const int64_t lo64 = ((int64_t)c * a.nwarps + warp) * a.per_warp;
    const int lo = (int)(lo64 < a.R ? lo64 : a.R);
    const int hi = (int)(lo64 + a.per_warp < a.R ? lo64 + a.per_warp : a.R);
    const int steps = warp < a.nwarps ? (hi - lo + 31) / 32 : 0;
    int32_t *mine = cnt + warp * B;
    int keep_key[kPlanKeep], keep_rank[kPlanKeep];  // of the steps this cluster writes
#pragma unroll
    for (int i = 0; i < kPlanKeep; ++i) keep_key[i] = -1, keep_rank[i] = 0;
    constexpr int kAhead = 8;
    for (int s0 = 0; s0 < steps; s0 += kAhead) {
        int keys[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) keys[i] = plan_key(a, lo + (s0 + i) * 32 + lane, hi);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (s0 + i >= steps) break;
            const int key = keys[i];
            unsigned same = __ballot_sync(0xffffffffu, key >= 0);
            for (int b = 0; b < a.bits; ++b) {
                const bool one = (key >> b) & 1;
                const unsigned v = __ballot_sync(0xffffffffu, one);
                same &= one ? v : ~v;
            }
            const int before = key >= 0 ? mine[key] : 0;
            __syncwarp();
            const int rank = before + __popc(same & ((1u << lane) - 1u));
            if (key >= 0 && (same >> lane) == 1u) mine[key] = rank + 1;  // its last lane
            __syncwarp();
            const int q = s0 + i - first_step;
#pragma unroll
            for (int t = 0; t < kPlanKeep; ++t)
                if (q == t && t < a.share) keep_key[t] = key, keep_rank[t] = rank;
        }
    }
    __syncthreads();

    // exclusive over this CTA's warps, 8 counts in flight; the totals go to the whole cluster
    for (int e = threadIdx.x; e < B; e += blockDim.x) {
        int run = 0;
        for (int w0 = 0; w0 < a.nwarps; w0 += 8) {
            int t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = w0 + i < a.nwarps ? cnt[(w0 + i) * B + e] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (w0 + i < a.nwarps) cnt[(w0 + i) * B + e] = run;
                run += t[i];
            }
        }
        tot[c * B + e] = run;
        for (int q = 0; q < C; ++q)
            if (q != c)
                asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(map_shared_rank(&tot[c * B + e], q)),
                             "r"(run)
                             : "memory");
    }
    if (C > 1) cluster_sync();
    else __syncthreads();

    // exclusive over the experts, chunks of blockDim.x experts
    int carry = 0;
    for (int e0 = 0; e0 < B; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        int all = 0, before = 0;
        if (e < B)
            for (int q = 0; q < C; ++q) {
                const int t = tot[q * B + e];
                all += t;
                if (q < c) before += t;
            }
        int inc = all;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += t;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        int w = lane < (int)(blockDim.x >> 5) ? wsum[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += t;
        }
        const int below = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
        const int start = carry + (warp > 0 ? below : 0) + inc - all;
        if (e < B) {
            base[e] = start + before;
            if (blockIdx.x == 0) a.offsets[e] = start;  // bucket E starts at the number of valid routes
        }
        carry += __shfl_sync(0xffffffffu, w, 31);
        __syncthreads();
    }

#pragma unroll
    for (int t = 0; t < kPlanKeep; ++t) {
        const int key = keep_key[t];
        if (key < 0) continue;
        const int r = lo + (first_step + t) * 32 + lane;
        const int row = base[key] + mine[key] + keep_rank[t];
        a.route_row[r] = key < a.E ? row : ~row;
        a.row_route[row] = key < a.E ? r : -1;
    }
}

// -------------------------------------------------------------------------------- row kernels
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float load(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 store(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
    static __device__ __forceinline__ float load(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half store(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<float> {
    static __device__ __forceinline__ float load(float v) { return v; }
    static __device__ __forceinline__ float store(float v) { return v; }
};

// V consecutive elements, moved as one access of V * sizeof(T) bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

// The row that route_row entry v names (complemented for a dropped route), or -1 for an entry
// no plan writes: such a route is skipped.
__device__ __forceinline__ int64_t row_of(int v, int64_t R) {
    const int64_t at = v < 0 ? ~v : v;
    return at < R ? at : -1;
}

struct RowArgs {
    const void *a, *b, *res;     // sort: x; sort_grad/unsort: rows; unsort_grad: gout, rows
    void *out, *out2;
    int64_t lda, ldb, ldres, ldout;  // elements
    const int32_t *route_row;
    const float *w;              // NULL: weights of one
    int M, k, H;
    int early;                   // unsort: all but the rows were complete before the kernel ahead began
};

// Sort: a unit is 32 * kSortVecs vectors of one token, read once and written k times.  The
// sorted rows are written in full and the token rows read once: the bytes the operator
// cannot do without, whatever the order (reading the rows in sorted order instead reads each
// token k times, from L2 at best).  8192 tokens x 8 routes x 2048 bf16: 46.2 us, 6.5 TB/s, 0.96 of
// the copy rate.
constexpr int kSortVecs = 4;
constexpr int kRowWarps = 8;

template <typename U>
__global__ void __launch_bounds__(32 * kRowWarps) token_sort_kernel(const RowArgs a, int nvec, int nchunk) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t units = (int64_t)a.M * nchunk;
    const int64_t stride = (int64_t)gridDim.x * kRowWarps;
    for (int64_t u = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5); u < units; u += stride) {
        const int64_t m = u / nchunk;
        const int v0 = (int)(u - m * nchunk) * (32 * kSortVecs) + lane;
        const U *src = static_cast<const U *>(a.a) + m * a.lda;
        const int row_l = lane < a.k ? a.route_row[m * a.k + lane] : 0;
        U v[kSortVecs];
#pragma unroll
        for (int i = 0; i < kSortVecs; ++i)
            if (v0 + 32 * i < nvec) v[i] = src[v0 + 32 * i];
        for (int j = 0; j < a.k; ++j) {
            const int row = __shfl_sync(0xffffffffu, row_l, j);
            const int64_t at = row_of(row, (int64_t)a.M * a.k);
            if (at < 0) continue;
            U *dst = static_cast<U *>(a.out) + at * a.ldout;
#pragma unroll
            for (int i = 0; i < kSortVecs; ++i)
                if (v0 + 32 * i < nvec) dst[v0 + 32 * i] = row < 0 ? U{} : v[i];
        }
    }
}

// Vectors a lane takes of a row at once in the forms for rows of any width, whose narrow loads
// in flight bound them: four of one element, two of two 16-bit ones, one of 16 bytes.
template <typename T, int V>
constexpr int kRowVecs = V * sizeof(T) >= 8 ? 1 : V == 1 ? 4 : 2;
// CTAs an SM of the unsort form, in a grid that fills the SMs once, and slots it loads at once.
// Four fp32 values of 8 slots at 2 CTAs left too few loads in flight: 4096 tokens x 32 routes x 1024
// fp32 160 us, with 4 slots at 4 CTAs 88.  (Eight 16-bit ones: 61 us this way, 138 at more CTAs.)
template <typename T, int V, int C>
constexpr int kUnsortCtas = C > 1 || V == 4 ? 4 : V * sizeof(T) >= 8 ? 2 : 3;
template <int V, int C>
constexpr int kUnsortSlots = C > 1 || V == 4 ? 4 : 8;

// Unsort, and with w == NULL and no residual the gradient of sort: a unit is 32 * C vectors of
// one token; the k rows' vectors are loaded kSlots at a time, then added in slot order.  The next
// unit's rows and weights are loaded meanwhile.  4096 tokens x 7 routes and a residual: 2047 bf16
// 63 us (with C = 1 and a warp a unit 93), 2046 bf16 49 (108), 2047 fp32 76 (101); 2048 tokens x
// 32 routes x 2048 bf16 61 us (137), 0.69 of the copy rate.  O: type of the residual and of out.
template <typename T, int V, int C, typename O = T>
__global__ void __launch_bounds__(32 * kRowWarps, kUnsortCtas<T, V, C>) token_unsort_kernel(const RowArgs a, int nvec, int nchunk) {
    constexpr int kSlots = kUnsortSlots<V, C>;
    using P = Pack<T, V>;
    using Q = Pack<O, V>;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t units = (int64_t)a.M * nchunk;
    const int64_t stride = (int64_t)gridDim.x * kRowWarps;
    int64_t u = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5), m_next = u / nchunk;
    int row_next = -1;
    float w_next = 1.0f;
    auto route = [&]() {
        if (u >= units || lane >= a.k) return;
        row_next = a.route_row[m_next * a.k + lane];
        if (a.w) w_next = a.w[m_next * a.k + lane];
    };
    route();
    while (u < units) {
        const int64_t m = m_next;
        const int v0 = (int)(u - m * nchunk) * (32 * C) + lane;
        const int row_l = row_of(row_next, (int64_t)a.M * a.k) < 0 ? -1 : row_next;
        const float w_l = w_next;
        u += stride, m_next = u / nchunk;
        route();
        float acc[C][V];
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[c][i] = 0.0f;
            if (a.res && v0 + 32 * c < nvec) {
                const Q r = *reinterpret_cast<const Q *>(static_cast<const O *>(a.res) + m * a.ldres + (int64_t)(v0 + 32 * c) * V);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[c][i] = Elem<O>::load(r.v[i]);
            }
        }
        for (int j0 = 0; j0 < a.k; j0 += kSlots) {
            P p[kSlots][C];
            int row[kSlots];
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                row[s] = __shfl_sync(0xffffffffu, row_l, (j0 + s) & 31);
                if (j0 + s >= a.k) row[s] = -1;
                const T *src = static_cast<const T *>(a.a) + (int64_t)row[s] * a.lda + (int64_t)v0 * V;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (row[s] >= 0 && v0 + 32 * c < nvec) p[s][c] = *reinterpret_cast<const P *>(src + 32 * c * V);
            }
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                const float w = __shfl_sync(0xffffffffu, w_l, (j0 + s) & 31);
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (row[s] >= 0 && v0 + 32 * c < nvec) {
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[c][i] = fmaf(w, Elem<T>::load(p[s][c].v[i]), acc[c][i]);
                    }
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (v0 + 32 * c < nvec) {
                Q o;
#pragma unroll
                for (int i = 0; i < V; ++i) o.v[i] = Elem<O>::store(acc[c][i]);
                *reinterpret_cast<Q *>(static_cast<O *>(a.out) + m * a.ldout + (int64_t)(v0 + 32 * c) * V) = o;
            }
    }
}

// Gradients of unsort: one CTA per token (grid-stride).  A thread holds C vectors of gout,
// multiplies them into the k gradient rows and adds their products with the k rows; the k dot
// products are then summed over the CTA in a fixed tree.  kSlots slots a pass.  4096 tokens x 7
// routes: 2047 bf16 64 us (with C = 1 114), 2047 fp32 92 (127); 2048 tokens x 32 routes x 2048 bf16
// 96 us, 0.83 of the copy rate.
constexpr int kGradThreads = 128;

template <typename T, int V, int C>
__global__ void __launch_bounds__(kGradThreads) token_unsort_grad_kernel(const RowArgs a, int nvec) {
    constexpr int kSlots = 8;
    using P = Pack<T, V>;
    __shared__ float part[kGradThreads / 32][kSlots];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        for (int j0 = 0; j0 < a.k; j0 += kSlots) {
            int row[kSlots], at[kSlots];
            float w[kSlots], dot[kSlots];
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                const bool on = j0 + s < a.k;
                row[s] = on ? a.route_row[m * a.k + j0 + s] : 0;
                at[s] = on ? (int)row_of(row[s], (int64_t)a.M * a.k) : -1;
                if (at[s] < 0) row[s] = -1;
                w[s] = on && a.w ? a.w[m * a.k + j0 + s] : 1.0f;
                dot[s] = 0.0f;
            }
            const T *g0 = static_cast<const T *>(a.a) + m * a.lda;
            for (int v0 = threadIdx.x; v0 < nvec; v0 += C * kGradThreads) {
                P g[C], y[kSlots][C];
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (v0 + c * kGradThreads < nvec) g[c] = *reinterpret_cast<const P *>(g0 + (int64_t)(v0 + c * kGradThreads) * V);
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    const T *src = static_cast<const T *>(a.b) + (int64_t)row[s] * a.ldb + (int64_t)v0 * V;
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        if (row[s] >= 0 && v0 + c * kGradThreads < nvec) y[s][c] = *reinterpret_cast<const P *>(src + c * kGradThreads * V);
                }
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    if (at[s] < 0) continue;
                    T *dst = static_cast<T *>(a.out) + (int64_t)at[s] * a.ldout + (int64_t)v0 * V;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        if (v0 + c * kGradThreads >= nvec) break;
                        P o;
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float gi = Elem<T>::load(g[c].v[i]);
                            if (row[s] >= 0) dot[s] = fmaf(gi, Elem<T>::load(y[s][c].v[i]), dot[s]);
                            o.v[i] = Elem<T>::store(row[s] >= 0 ? w[s] * gi : 0.0f);
                        }
                        *reinterpret_cast<P *>(dst + c * kGradThreads * V) = o;
                    }
                }
            }
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot[s] += __shfl_xor_sync(0xffffffffu, dot[s], d);
                if (lane == 0) part[warp][s] = dot[s];
            }
            __syncthreads();
            if (threadIdx.x < kSlots && j0 + (int)threadIdx.x < a.k) {
                float t = 0.0f;
                for (int q = 0; q < kGradThreads / 32; ++q) t += part[q][threadIdx.x];
                static_cast<float *>(a.out2)[m * a.k + j0 + threadIdx.x] = t;
            }
            __syncthreads();
        }
    }
}

// ------------------------------------------------------------------- row kernels, 16-byte rows
// The same two operators where every row is whole 16-byte pieces.  What bounds the form above
// is latency: a warp loads its indices, then its rows, then stores, and holds one unit's rows in
// registers.  Here each lane copies its own pieces of the next kDepth units into its own slots
// of shared memory (cp.async), so a warp has kDepth units in flight and no thread waits for
// another.  The arithmetic and its order per element are those of the form above.  8192 tokens x
// 8 routes x 2048 bf16 (form above): unsort 54.9 us, 0.90 of the copy rate (75); without weights
// and residual, as the gradient of sort, 47.5 us, 0.94 (64); one token 2.4 us (2.3).
constexpr int kRingWarps = 8;
// Shared memory of a CTA, whatever part its slots fill: three CTAs an SM, in a grid that fills
// the SMs once.  Every such launch asks for the same size: with sizes of their own, a grid that
// starts while another drains found holes that fit two CTAs on a few SMs, and the third ran
// after all others (gradients of 8192 tokens 226 against 168 us).
constexpr int kRingBytes = 74 * 1024;
constexpr int kRingCtas = 3;
constexpr int kRingSlots = 8;  // slots of the gradient's dot products
constexpr int kRingSmem = kRingBytes + 2 * kRingWarps * kRingSlots * 4;  // and their partial sums

// One unit of the ring: the k rows' pieces, then the token's own (residual or gradient).
struct RingUnit {
    int64_t m;
    int vi;  // this lane's 16-byte piece of the row
};

// O: the type of the token's own piece, as many elements as a piece of the rows.
template <typename T, typename O = T>
__device__ __forceinline__ void ring_issue(const RowArgs &a, const void *rows, int64_t ldrows, const void *own,
                                           int64_t ldown, const RingUnit &u, int nvec, int row_l, uint4 *slot) {
    constexpr int n = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
    const bool in = u.vi < nvec;
    for (int j = 0; j < a.k; ++j) {
        const int row = __shfl_sync(0xffffffffu, row_l, j);
        // a dropped route's slot is filled with zeros, from no address of its own
        if (in)
            cp_async_16_zfill(slot + j * 32 + lane,
                              static_cast<const T *>(rows) + (row >= 0 ? (int64_t)row * ldrows + (int64_t)u.vi * n : 0),
                              row >= 0 ? 16u : 0u);
    }
    if (own && in) {
        const O *src = static_cast<const O *>(own) + u.m * ldown + (int64_t)u.vi * n;
        if constexpr (sizeof(O) == sizeof(T)) cp_async_16(slot + a.k * 32 + lane, src);
        else cp_async_8(slot + a.k * 32 + lane, src);
    }
}

// One 16-byte piece as fp32.
template <typename T>
__device__ __forceinline__ void ring_load(const uint4 *p, float (&v)[16 / sizeof(T)]) {
    const uint4 u = *p;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
    } else {
        const T *t = reinterpret_cast<const T *>(&u);
#pragma unroll
        for (int i = 0; i < (int)(16 / sizeof(T)); ++i) v[i] = Elem<T>::load(t[i]);
    }
}

// A token's own piece of n elements of another type than the rows'.
template <typename O, int n>
__device__ __forceinline__ void ring_load_own(const uint4 *p, float (&v)[n]) {
    const Pack<O, n> o = *reinterpret_cast<const Pack<O, n> *>(p);
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = Elem<O>::load(o.v[i]);
}

// route_row entry of lane j < k for token m, -1 for a dropped or unknown row.
__device__ __forceinline__ int ring_row(const RowArgs &a, int64_t m) {
    const int lane = threadIdx.x & 31;
    if (lane >= a.k) return -1;
    const int32_t *at = a.route_row + m * a.k + lane;
    const int v = a.early ? __ldcg(at) : *at;
    return row_of(v, (int64_t)a.M * a.k) < 0 ? -1 : v;
}

// A warp's sequence of units: chunks q, q + wpt, ... of tokens m, m + step, ... (no
// division: the 64-bit ones were a tenth of the kernel's time, 81 against 73 us).
struct RingCursor {
    int64_t m;
    int c;
    __device__ __forceinline__ void advance(int q, int wpt, int nchunk, int64_t step) {
        c += wpt;
        if (c >= nchunk) c = q, m += step;
    }
};

// O: type of the residual and of out.
template <typename T, typename O, int kDepth>
__global__ void __launch_bounds__(32 * kRingWarps) token_unsort_ring_kernel(const RowArgs a, int nvec, int nchunk, int wpt) {
    constexpr int n = 16 / sizeof(T);
    using P = Pack<O, n>;
    extern __shared__ uint4 ring[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (a.k + (a.res ? 1 : 0)) * 32;
    uint4 *mine = ring + (size_t)warp * kDepth * per;
    const int q = warp % wpt, tokens = kRingWarps / wpt;
    const int64_t step = (int64_t)gridDim.x * tokens;
    RingCursor now{(int64_t)blockIdx.x * tokens + warp / wpt, q}, ahead = now;
    if (!a.early) pdl_wait();

    // rows of the token the copies are at; weights of the one the sums are at and of the next
    int row_a = -1;
    float w = 0.0f, w_n = 0.0f;
    // a dropped route's weight is zero, whatever the caller's says
    auto weight = [&](int64_t m) {
        if (ring_row(a, m) < 0) return 0.0f;
        if (!a.w) return 1.0f;
        const float *at = a.w + m * a.k + lane;
        return a.early ? __ldcg(at) : *at;
    };
    if (now.m < a.M) {
        row_a = ring_row(a, now.m);
        w = weight(now.m);
        if (now.m + step < a.M) w_n = weight(now.m + step);
    }
    if (a.early) pdl_wait();
    pdl_launch_dependents();
    int slot_in = 0, slot_out = 0;
    auto issue = [&]() {
        if (ahead.m < a.M) {
            ring_issue<T, O>(a, a.a, a.lda, a.res, a.ldres, RingUnit{ahead.m, ahead.c * 32 + lane}, nvec, row_a, mine + slot_in * per);
            const int64_t m = ahead.m;
            ahead.advance(q, wpt, nchunk, step);
            if (ahead.m != m) row_a = ahead.m < a.M ? ring_row(a, ahead.m) : -1;
        }
        cp_async_commit();
        if (++slot_in == kDepth) slot_in = 0;
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) issue();
    while (now.m < a.M) {
        cp_async_wait_group<kDepth - 1>();
        const int vi = now.c * 32 + lane;
        const uint4 *slot = mine + slot_out * per;
        const bool in = vi < nvec;
        float acc[n];
#pragma unroll
        for (int i = 0; i < n; ++i) acc[i] = 0.0f;
        if (a.res && in) {
            if constexpr (std::is_same<T, O>::value) ring_load<T>(slot + a.k * 32 + lane, acc);
            else ring_load_own<O>(slot + a.k * 32 + lane, acc);
        }
#pragma unroll 8
        for (int j = 0; j < a.k; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            float v[n];
            ring_load<T>(slot + j * 32 + lane, v);
#pragma unroll
            for (int i = 0; i < n; i += 2) ffma2(acc[i], acc[i + 1], wj, v[i], v[i + 1]);
        }
        if (in) {
            P o;
#pragma unroll
            for (int i = 0; i < n; ++i) o.v[i] = Elem<O>::store(acc[i]);
            *reinterpret_cast<P *>(static_cast<O *>(a.out) + now.m * a.ldout + (int64_t)vi * n) = o;
        }
        if (++slot_out == kDepth) slot_out = 0;
        issue();
        const int64_t m = now.m;
        now.advance(q, wpt, nchunk, step);
        if (now.m != m) {
            w = w_n;
            if (now.m + step < a.M) w_n = weight(now.m + step);
        }
    }
    cp_async_wait_all();
}

// One CTA per token (grid-stride): warp q takes chunks q, q + 8, ... of the row, a running
// sequence of units over all its tokens; the k <= 8 products are summed over the lanes, then
// over the warps, in fixed trees.  8192 tokens x 8 routes x 2048 bf16: 88.9 us, 0.94 of the copy
// rate (form above 100); one token 3.5 us (2.9).
template <typename T, int kDepth>
__global__ void __launch_bounds__(32 * kRingWarps) token_unsort_grad_ring_kernel(const RowArgs a, int nvec, int nchunk) {
    constexpr int n = 16 / sizeof(T);
    using P = Pack<T, n>;
    extern __shared__ uint4 ring[];
    float (*part)[kRingWarps][kRingSlots] = reinterpret_cast<float (*)[kRingWarps][kRingSlots]>(ring + kRingBytes / 16);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (a.k + 1) * 32;
    uint4 *mine = ring + (size_t)warp * kDepth * per;
    const int mychunks = nchunk > warp ? (nchunk - warp + kRingWarps - 1) / kRingWarps : 0;
    pdl_wait();
    pdl_launch_dependents();

    // the unit `steps` after (m, c)
    struct Cursor {
        int64_t m;
        int c;
    };
    auto advance = [&](Cursor &x) {
        if (++x.c == mychunks) x.c = 0, x.m += gridDim.x;
    };
    auto unit = [&](const Cursor &x) { return RingUnit{x.m, (warp + x.c * kRingWarps) * 32 + lane}; };
    Cursor ahead{(int64_t)blockIdx.x, 0};
    int slot_in = 0, slot_out = 0;
    int row_ahead = -1;
    if (mychunks > 0 && ahead.m < a.M) row_ahead = ring_row(a, ahead.m);
    auto issue = [&]() {
        if (mychunks > 0 && ahead.m < a.M) {
            ring_issue<T>(a, a.b, a.ldb, a.a, a.lda, unit(ahead), nvec, row_ahead, mine + slot_in * per);
            const int64_t m = ahead.m;
            advance(ahead);
            if (ahead.m != m) row_ahead = ahead.m < a.M ? ring_row(a, ahead.m) : -1;
        }
        cp_async_commit();
        if (++slot_in == kDepth) slot_in = 0;
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) issue();

    int parity = 0;
    int v_next = 0;
    float w_next = 1.0f;
    if (lane < a.k && (int64_t)blockIdx.x < a.M) {
        v_next = a.route_row[(int64_t)blockIdx.x * a.k + lane];
        if (a.w) w_next = a.w[(int64_t)blockIdx.x * a.k + lane];
    }
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, parity ^= 1) {
        const int v_l = v_next;
        const float w_l = w_next;
        const int64_t mn = m + gridDim.x;
        if (lane < a.k && mn < a.M) {
            v_next = a.route_row[mn * a.k + lane];
            if (a.w) w_next = a.w[mn * a.k + lane];
        }
        float dot[kRingSlots];
#pragma unroll
        for (int s = 0; s < kRingSlots; ++s) dot[s] = 0.0f;
        for (int c = 0; c < mychunks; ++c) {
            cp_async_wait_group<kDepth - 1>();
            const int vi = (warp + c * kRingWarps) * 32 + lane;
            const uint4 *slot = mine + slot_out * per;
            const bool in = vi < nvec;
            float g[n];
            ring_load<T>(slot + a.k * 32 + lane, g);
#pragma unroll
            for (int s = 0; s < kRingSlots; ++s) {
                if (s >= a.k) break;
                const int v = __shfl_sync(0xffffffffu, v_l, s);
                const float w = __shfl_sync(0xffffffffu, w_l, s);
                const int64_t at = row_of(v, (int64_t)a.M * a.k);
                if (in && at >= 0) {
                    P o;
                    if (v >= 0) {
                        float y[n];
                        ring_load<T>(slot + s * 32 + lane, y);
#pragma unroll
                        for (int i = 0; i < n; ++i) {
                            dot[s] = fmaf(g[i], y[i], dot[s]);
                            o.v[i] = Elem<T>::store(w * g[i]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < n; ++i) o.v[i] = Elem<T>::store(0.0f);
                    }
                    *reinterpret_cast<P *>(static_cast<T *>(a.out) + at * a.ldout + (int64_t)vi * n) = o;
                }
            }
            if (++slot_out == kDepth) slot_out = 0;
            issue();
        }
        // 8 sums over 32 lanes: halves exchanged until a lane holds one slot, then added
#pragma unroll
        for (int h = 4; h >= 1; h >>= 1) {
            const bool up = lane & (4 * h);
#pragma unroll
            for (int i = 0; i < h; ++i) {
                const float send = up ? dot[i] : dot[i + h];
                const float keep = up ? dot[i + h] : dot[i];
                dot[i] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * h);
            }
        }
        float t = dot[0];
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        // lane bits 4, 3, 2 chose the slot's bits 2, 1, 0
        if ((lane & 3) == 0) part[parity][warp][lane >> 2] = t;
        __syncthreads();
        if ((int)threadIdx.x < a.k) {
            float sum = 0.0f;
            for (int q = 0; q < kRingWarps; ++q) sum += part[parity][q][threadIdx.x];
            static_cast<float *>(a.out2)[m * a.k + threadIdx.x] = sum;
        }
    }
    cp_async_wait_all();
}

// ----------------------------------------------------------------------------------- launchers
static int64_t cap_grid(int64_t ctas, int per_sm) {
    const int64_t most = (int64_t)num_sms() * per_sm;
    return ctas < most ? (ctas > 0 ? ctas : 1) : most;
}

cudaError_t launch_token_plan(const int32_t *ids, int M, int k, int E, int32_t *offsets,
                              int32_t *row_route, int32_t *route_row, cudaStream_t stream) {
    PlanArgs a{ids, offsets, row_route, route_row, M * k, E, 0, 0, 0, 1, kPlanKeep};
    while ((1 << a.bits) <= E) ++a.bits;
    // runs of 128 routes a warp where there are enough of them, up to 8 CTAs of 32 warps; then
    // runs of up to 1024 routes in 8 clusters that each write 4 of a run's 32 steps, and past
    // 262,144 routes more clusters
    const int64_t groups = ((int64_t)a.R + 127) / 128;
    while (a.C < kPlanMaxCluster && groups > 32 * a.C) a.C *= 2;
    const int64_t per_cta = (groups + a.C - 1) / a.C;
    a.nwarps = (int)(per_cta < 1 ? 1 : per_cta > 32 ? 32 : per_cta);
    const int64_t warps = (int64_t)a.C * a.nwarps, per_warp = ((int64_t)a.R + warps - 1) / warps;
    a.per_warp = (int)((per_warp + 31) / 32 * 32);
    const int steps = a.per_warp / 32;
    a.share = steps <= kPlanMaxShares ? 1 : (steps + kPlanMaxShares - 1) / kPlanMaxShares;
    if (a.share > kPlanKeep) a.share = kPlanKeep;
    const int clusters = steps > 0 ? (steps + a.share - 1) / a.share : 1;
    int threads = a.nwarps * 32;
    const int want = (E + 1 + 31) / 32 * 32;
    if (threads < want) threads = want < 1024 ? want : 1024;
    const size_t smem = (size_t)(a.nwarps + kPlanMaxCluster + 1) * (E + 1) * 4;
    cudaError_t err = ensure_smem((const void *)token_plan_kernel, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(dim3(a.C * clusters), dim3(threads), smem, stream, attrs, a.C > 1 ? a.C : 0);
    return cudaLaunchKernelEx(&cfg, token_plan_kernel, a);
}

// The widest access (bytes, one of 16, 4, elem) that every pointer, row pitch and the row
// length allow.
static int vec_bytes(const RowArgs &a, int elem) {
    uint64_t bits = (uint64_t)a.H * elem;
    const void *ptrs[4] = {a.a, a.b, a.res, a.out};
    const int64_t lds[4] = {a.lda, a.ldb, a.ldres, a.ldout};
    for (int i = 0; i < 4; ++i)
        if (ptrs[i]) bits |= reinterpret_cast<uintptr_t>(ptrs[i]) | (uint64_t)(lds[i] * elem);
    return bits % 16 == 0 ? 16 : (bits % 4 == 0 ? 4 : elem);
}

template <typename U>
static cudaError_t sort_as(RowArgs a, int elem, cudaStream_t stream) {
    const int per = (int)sizeof(U) / elem;  // elements per access
    a.lda /= per;
    a.ldout /= per;
    const int nvec = a.H / per;
    const int nchunk = (nvec + 32 * kSortVecs - 1) / (32 * kSortVecs);
    const int64_t ctas = ((int64_t)a.M * nchunk + kRowWarps - 1) / kRowWarps;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)cap_grid(ctas, 64)), dim3(32 * kRowWarps), 0, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, token_sort_kernel<U>, a, nvec, nchunk);
}

template <typename T, int V, int C, typename O>
static cudaError_t unsort_vecs(const RowArgs &a, cudaStream_t stream) {
    const int nvec = a.H / V;
    const int nchunk = (nvec + 32 * C - 1) / (32 * C);
    const int64_t ctas = ((int64_t)a.M * nchunk + kRowWarps - 1) / kRowWarps;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)cap_grid(ctas, kUnsortCtas<T, V, C>)), dim3(32 * kRowWarps), 0, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, token_unsort_kernel<T, V, C, O>, a, nvec, nchunk);
}

// One vector a lane while every warp then has one unit at most (one token of 2047 bf16 2.2 us,
// with four 3.3).
template <typename T, int V, typename O = T>
static cudaError_t unsort_as(const RowArgs &a, cudaStream_t stream) {
    const int64_t units = (int64_t)a.M * ((a.H / V + 31) / 32);
    if (units <= (int64_t)num_sms() * kUnsortCtas<T, V, 1> * kRowWarps) return unsort_vecs<T, V, 1, O>(a, stream);
    return unsort_vecs<T, V, kRowVecs<T, V>, O>(a, stream);
}

template <typename T, int V, int C>
static cudaError_t unsort_grad_vecs(const RowArgs &a, cudaStream_t stream) {
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)cap_grid(a.M, 64)), dim3(kGradThreads), 0, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, token_unsort_grad_kernel<T, V, C>, a, a.H / V);
}

// As many vectors a thread as cover the row: more only take registers from other CTAs (4096 tokens
// x 7 routes: 65 bf16 11.4 us, with four vectors 13.9; 129 fp32 17.4 with two, 22.6).
template <typename T, int V>
static cudaError_t unsort_grad_as(const RowArgs &a, cudaStream_t stream) {
    constexpr int most = kRowVecs<T, V>;
    const int need = (a.H / V + kGradThreads - 1) / kGradThreads;
    if (need == 1) return unsort_grad_vecs<T, V, 1>(a, stream);
    if (need == 2) return unsort_grad_vecs<T, V, most < 2 ? most : 2>(a, stream);
    return unsort_grad_vecs<T, V, most>(a, stream);
}

// Whether `depth` units of `rows` pieces a warp fit a CTA's slots.
static bool ring_fits(int rows, int depth) { return kRingWarps * depth * rows * 512 <= kRingBytes; }

// Units in flight a warp: as many of 8, 4, 2, 1 as fit.
static int ring_depth(int rows) {
    int d = 8;
    while (d > 1 && !ring_fits(rows, d)) d /= 2;
    return d;
}

template <typename T, typename O, int kDepth>
static cudaError_t unsort_ring_as(const RowArgs &a, cudaStream_t stream) {
    if (!ring_fits(a.k + (a.res ? 1 : 0), kDepth)) return cudaErrorInvalidValue;
    const int nvec = a.H / (16 / (int)sizeof(T)), nchunk = (nvec + 31) / 32;
    const auto fn = token_unsort_ring_kernel<T, O, kDepth>;
    cudaError_t err = ensure_smem((const void *)fn, kRingSmem);
    if (err != cudaSuccess) return err;
    int wpt = 1;  // warps a token
    while (wpt < kRingWarps && wpt * 2 <= nchunk) wpt *= 2;
    const int64_t ctas = ((int64_t)a.M * wpt + kRingWarps - 1) / kRingWarps;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)cap_grid(ctas, kRingCtas)), dim3(32 * kRingWarps), kRingSmem, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, fn, a, nvec, nchunk, wpt);
}

template <typename T, int kDepth>
static cudaError_t unsort_grad_ring_as(const RowArgs &a, cudaStream_t stream) {
    if (!ring_fits(a.k + 1, kDepth)) return cudaErrorInvalidValue;
    const int nvec = a.H / (16 / (int)sizeof(T)), nchunk = (nvec + 31) / 32;
    const auto fn = token_unsort_grad_ring_kernel<T, kDepth>;
    cudaError_t err = ensure_smem((const void *)fn, kRingSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)cap_grid(a.M, kRingCtas)), dim3(32 * kRingWarps), kRingSmem, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, fn, a, nvec, nchunk);
}

template <typename T, typename O = T>
static cudaError_t unsort_ring(const RowArgs &a, cudaStream_t stream) {
    switch (ring_depth(a.k + (a.res ? 1 : 0))) {
        case 8: return unsort_ring_as<T, O, 8>(a, stream);
        case 4: return unsort_ring_as<T, O, 4>(a, stream);
        case 2: return unsort_ring_as<T, O, 2>(a, stream);
        default: return unsort_ring_as<T, O, 1>(a, stream);
    }
}

template <typename T>
static cudaError_t unsort_grad_ring(const RowArgs &a, cudaStream_t stream) {
    switch (ring_depth(a.k + 1)) {
        case 8: return unsort_grad_ring_as<T, 8>(a, stream);
        case 4: return unsort_grad_ring_as<T, 4>(a, stream);
        default: return unsort_grad_ring_as<T, 2>(a, stream);
    }
}

cudaError_t launch_token_sort(const void *x, int64_t ldx, int elem, int M, int k, int H,
                              const int32_t *route_row, void *rows, int64_t ldr, cudaStream_t stream) {
    RowArgs a{};
    a.a = x, a.out = rows, a.lda = ldx, a.ldout = ldr;
    a.route_row = route_row, a.M = M, a.k = k, a.H = H;
    switch (vec_bytes(a, elem)) {
        case 16: return sort_as<uint4>(a, elem, stream);
        case 4: return sort_as<uint32_t>(a, elem, stream);
        default: return sort_as<uint16_t>(a, elem, stream);
    }
}

// Calls F<T, V>(args, stream) for the element type and an access of vb bytes; 16-byte rows go to
// the ring forms where they fit (unsort up to 17 slots and a residual, its gradient up to 8).
#define MOE_ROW_DISPATCH(F, RING, takes)                                                             \
    const int vb = vec_bytes(a, dtype == MOE_DT_F32 ? 4 : 2);                                        \
    if (vb == 16 && (takes)) {                                                                       \
        if (dtype == MOE_DT_F32) return RING<float>(a, stream);                                      \
        return dtype == MOE_DT_F16 ? RING<__half>(a, stream) : RING<__nv_bfloat16>(a, stream);       \
    }                                                                                                \
    if (dtype == MOE_DT_F32) return vb == 16 ? F<float, 4>(a, stream) : F<float, 1>(a, stream);      \
    if (dtype == MOE_DT_F16)                                                                         \
        return vb == 16 ? F<__half, 8>(a, stream)                                                    \
                        : vb == 4 ? F<__half, 2>(a, stream) : F<__half, 1>(a, stream);               \
    return vb == 16 ? F<__nv_bfloat16, 8>(a, stream)                                                 \
                    : vb == 4 ? F<__nv_bfloat16, 2>(a, stream) : F<__nv_bfloat16, 1>(a, stream);

static RowArgs unsort_args(const void *rows, int64_t ldr, int M, int k, int H, const int32_t *route_row,
                           const float *w, const void *residual, int64_t ldres, void *out, int64_t ldo, bool early) {
    RowArgs a{};
    a.early = early;
    a.a = rows, a.res = residual, a.out = out, a.lda = ldr, a.ldres = ldres, a.ldout = ldo;
    a.route_row = route_row, a.w = w, a.M = M, a.k = k, a.H = H;
    return a;
}

cudaError_t launch_token_unsort(const void *rows, int64_t ldr, int dtype, int M, int k, int H,
                                const int32_t *route_row, const float *w, const void *residual,
                                int64_t ldres, void *out, int64_t ldo, bool early, cudaStream_t stream) {
    const RowArgs a = unsort_args(rows, ldr, M, k, H, route_row, w, residual, ldres, out, ldo, early);
    MOE_ROW_DISPATCH(unsort_as, unsort_ring, ring_fits(k + (residual ? 1 : 0), 1))
}

cudaError_t launch_token_unsort_f32(const float *rows, int M, int k, int H, const int32_t *route_row, const float *w,
                                    const __nv_bfloat16 *residual, __nv_bfloat16 *out, bool early, cudaStream_t stream) {
    const RowArgs a = unsort_args(rows, H, M, k, H, route_row, w, residual, H, out, H, early);
    if (ring_fits(k + (residual ? 1 : 0), 1)) return unsort_ring<float, __nv_bfloat16>(a, stream);
    return unsort_as<float, 4, __nv_bfloat16>(a, stream);
}

cudaError_t launch_token_unsort_grad(const void *gout, int64_t ldo, const void *rows, int64_t ldr,
                                     int dtype, int M, int k, int H, const int32_t *route_row,
                                     const float *w, void *grows, int64_t ldg, float *gw,
                                     cudaStream_t stream) {
    RowArgs a{};
    a.a = gout, a.b = rows, a.out = grows, a.out2 = gw, a.lda = ldo, a.ldb = ldr, a.ldout = ldg;
    a.route_row = route_row, a.w = w, a.M = M, a.k = k, a.H = H;
    MOE_ROW_DISPATCH(unsort_grad_as, unsort_grad_ring, k <= kRingSlots)
}

}  // namespace moe
