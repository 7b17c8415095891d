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
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {

// ------------------------------------------------------------------------------------- plan
// One cluster of C CTAs.  Each warp takes a contiguous run of routes and counts them per
// expert in its own row of shared memory, 32 routes a step: the lanes that share an expert
// find each other with match.any, so a route's rank inside its warp's run needs no atomics
// and follows r.  Two scans (over the warps of a CTA, then over the CTAs of the cluster,
// through distributed shared memory) and one over the experts turn ranks into rows.
// Dropped routes use bucket E, which follows the last expert.
constexpr int kPlanMaxCluster = 8;
constexpr int kPlanKeep = 4;  // steps whose ranks stay in registers; longer runs park them in route_row

struct PlanArgs {
    const int32_t *ids;
    int32_t *offsets, *row_route, *route_row;
    int R, E;
    int per_warp;  // routes per warp, a multiple of 32
    int nwarps;    // warps per CTA that hold routes
};

__global__ void __launch_bounds__(1024) token_plan_kernel(const PlanArgs a) {
    extern __shared__ int32_t sm[];
    const int B = a.E + 1;                       // buckets
    int32_t *cnt = sm;                           // [nwarps][B]
    int32_t *tot = cnt + a.nwarps * B;           // [C][B] every CTA's totals
    int32_t *base = tot + kPlanMaxCluster * B;   // [B]
    __shared__ int32_t wsum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x, C = gridDim.x;

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
    int keep_key[kPlanKeep], keep_rank[kPlanKeep];
    for (int s0 = 0; s0 < steps; s0 += kPlanKeep) {
#pragma unroll
        for (int i = 0; i < kPlanKeep; ++i) {
            const int r = lo + (s0 + i) * 32 + lane;
            const int id = r < hi ? a.ids[r] : 0;
            keep_key[i] = r < hi ? ((uint32_t)id < (uint32_t)a.E ? id : a.E) : -1;
        }
#pragma unroll
        for (int i = 0; i < kPlanKeep; ++i) {
            if (s0 + i >= steps) break;
            const int key = keep_key[i];
            const unsigned same = __match_any_sync(0xffffffffu, key);
            const int before = key >= 0 ? mine[key] : 0;
            __syncwarp();
            const int rank = before + __popc(same & ((1u << lane) - 1u));
            if (key >= 0 && lane == 31 - __clz(same)) mine[key] = rank + 1;
            __syncwarp();
            keep_rank[i] = rank;
            if (steps > kPlanKeep && key >= 0) a.route_row[lo + (s0 + i) * 32 + lane] = rank;
        }
    }
    __syncthreads();

    // exclusive over this CTA's warps; the totals go to every CTA of the cluster
    for (int e = threadIdx.x; e < B; e += blockDim.x) {
        int run = 0;
        for (int w = 0; w < a.nwarps; ++w) {
            const int t = cnt[w * B + e];
            cnt[w * B + e] = run;
            run += t;
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
        int off = carry, chunk = 0;
        for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
            const int t = wsum[w];
            if (w < warp) off += t;
            chunk += t;
        }
        const int start = off + inc - all;
        if (e < B) {
            base[e] = start + before;
            if (c == 0) a.offsets[e] = start;  // bucket E starts at the number of valid routes
        }
        carry += chunk;
        __syncthreads();
    }

    for (int s0 = 0; s0 < steps; s0 += kPlanKeep) {
        if (steps > kPlanKeep) {
#pragma unroll
            for (int i = 0; i < kPlanKeep; ++i) {
                const int r = lo + (s0 + i) * 32 + lane;
                const int id = r < hi ? a.ids[r] : 0;
                keep_key[i] = r < hi ? ((uint32_t)id < (uint32_t)a.E ? id : a.E) : -1;
                keep_rank[i] = r < hi ? a.route_row[r] : 0;
            }
        }
#pragma unroll
        for (int i = 0; i < kPlanKeep; ++i) {
            if (s0 + i >= steps) break;
            const int key = keep_key[i];
            if (key < 0) continue;
            const int r = lo + (s0 + i) * 32 + lane;
            const int row = base[key] + mine[key] + keep_rank[i];
            a.route_row[r] = key < a.E ? row : ~row;
            a.row_route[row] = key < a.E ? r : -1;
        }
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
};

// Sort: a unit is 32 * kSortVecs vectors of one token, read once and written k times.  The
// sorted rows are written in full and the token rows read once: the bytes the operator
// cannot do without, whatever the order (reading the rows in sorted order instead reads each
// token k times, from L2 at best).
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

// Unsort, and with w == NULL and no residual the gradient of sort: a unit is 32 vectors of
// one token; the k rows' vectors are loaded kSlots at a time, then added in slot order.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kRowWarps) token_unsort_kernel(const RowArgs a, int nvec, int nchunk) {
    constexpr int kSlots = 8;
    using P = Pack<T, V>;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t units = (int64_t)a.M * nchunk;
    const int64_t stride = (int64_t)gridDim.x * kRowWarps;
    for (int64_t u = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5); u < units; u += stride) {
        const int64_t m = u / nchunk;
        const int vi = (int)(u - m * nchunk) * 32 + lane;
        const bool in = vi < nvec;
        const int row_l = lane < a.k ? a.route_row[m * a.k + lane] : -1;
        const float w_l = a.w && lane < a.k ? a.w[m * a.k + lane] : 1.0f;
        float acc[V];
        if (a.res && in) {
            const P r = *reinterpret_cast<const P *>(static_cast<const T *>(a.res) + m * a.ldres + (int64_t)vi * V);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = Elem<T>::load(r.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        }
        for (int j0 = 0; j0 < a.k; j0 += kSlots) {
            P p[kSlots];
            int row[kSlots];
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                row[s] = __shfl_sync(0xffffffffu, row_l, (j0 + s) & 31);
                if (j0 + s >= a.k || !in || row_of(row[s], (int64_t)a.M * a.k) < 0) row[s] = -1;
                if (row[s] >= 0)
                    p[s] = *reinterpret_cast<const P *>(static_cast<const T *>(a.a) + (int64_t)row[s] * a.lda + (int64_t)vi * V);
            }
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                const float w = __shfl_sync(0xffffffffu, w_l, (j0 + s) & 31);
                if (row[s] >= 0) {
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = fmaf(w, Elem<T>::load(p[s].v[i]), acc[i]);
                }
            }
        }
        if (in) {
            P o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.v[i] = Elem<T>::store(acc[i]);
            *reinterpret_cast<P *>(static_cast<T *>(a.out) + m * a.ldout + (int64_t)vi * V) = o;
        }
    }
}

// Gradients of unsort: one CTA per token (grid-stride).  A thread holds one vector of gout,
// multiplies it into the k gradient rows and adds its products with the k rows; the k dot
// products are then summed over the CTA in a fixed tree.  kSlots slots a pass.
constexpr int kGradThreads = 128;

template <typename T, int V>
__global__ void __launch_bounds__(kGradThreads) token_unsort_grad_kernel(const RowArgs a, int nvec) {
    constexpr int kSlots = 8;
    using P = Pack<T, V>;
    __shared__ float part[kGradThreads / 32][kSlots];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        for (int j0 = 0; j0 < a.k; j0 += kSlots) {
            int row[kSlots];
            int64_t at[kSlots];
            float w[kSlots], dot[kSlots];
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                const bool on = j0 + s < a.k;
                row[s] = on ? a.route_row[m * a.k + j0 + s] : 0;
                at[s] = row_of(row[s], (int64_t)a.M * a.k);
                if (at[s] < 0) row[s] = -1;
                w[s] = on && a.w ? a.w[m * a.k + j0 + s] : 1.0f;
                dot[s] = 0.0f;
            }
            const T *g0 = static_cast<const T *>(a.a) + m * a.lda;
            for (int vi = threadIdx.x; vi < nvec; vi += kGradThreads) {
                const P g = *reinterpret_cast<const P *>(g0 + (int64_t)vi * V);
                P y[kSlots];
#pragma unroll
                for (int s = 0; s < kSlots; ++s)
                    if (j0 + s < a.k && row[s] >= 0)
                        y[s] = *reinterpret_cast<const P *>(static_cast<const T *>(a.b) + (int64_t)row[s] * a.ldb + (int64_t)vi * V);
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    if (j0 + s >= a.k) break;
                    P o;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float gi = Elem<T>::load(g.v[i]);
                        if (row[s] >= 0) dot[s] = fmaf(gi, Elem<T>::load(y[s].v[i]), dot[s]);
                        o.v[i] = Elem<T>::store(row[s] >= 0 ? w[s] * gi : 0.0f);
                    }
                    if (at[s] >= 0)
                        *reinterpret_cast<P *>(static_cast<T *>(a.out) + at[s] * a.ldout + (int64_t)vi * V) = o;
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

// ----------------------------------------------------------------------------------- launchers
static int64_t cap_grid(int64_t ctas, int per_sm) {
    const int64_t most = (int64_t)num_sms() * per_sm;
    return ctas < most ? (ctas > 0 ? ctas : 1) : most;
}

cudaError_t launch_token_plan(const int32_t *ids, int M, int k, int E, int32_t *offsets,
                              int32_t *row_route, int32_t *route_row, cudaStream_t stream) {
    PlanArgs a{ids, offsets, row_route, route_row, M * k, E, 0, 0};
    // 128 routes a warp where there are enough of them, up to 8 CTAs of 32 warps
    const int64_t groups = ((int64_t)a.R + 127) / 128;
    int C = 1;
    while (C < kPlanMaxCluster && groups > 32 * C) C *= 2;
    const int64_t per_cta = (groups + C - 1) / C;
    a.nwarps = (int)(per_cta < 1 ? 1 : per_cta > 32 ? 32 : per_cta);
    const int64_t per_warp = ((int64_t)a.R + (int64_t)C * a.nwarps - 1) / ((int64_t)C * a.nwarps);
    a.per_warp = (int)((per_warp + 31) / 32 * 32);
    int threads = a.nwarps * 32;
    const int want = (E + 1 + 31) / 32 * 32;
    if (threads < want) threads = want < 1024 ? want : 1024;
    const size_t smem = (size_t)(a.nwarps + kPlanMaxCluster + 1) * (E + 1) * 4;
    cudaError_t err = ensure_smem((const void *)token_plan_kernel, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(dim3(C), dim3(threads), smem, stream, attrs, C > 1 ? C : 0);
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

template <typename T, int V>
static cudaError_t unsort_as(const RowArgs &a, cudaStream_t stream) {
    const int nvec = a.H / V;
    const int nchunk = (nvec + 31) / 32;
    const int64_t ctas = ((int64_t)a.M * nchunk + kRowWarps - 1) / kRowWarps;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)cap_grid(ctas, 64)), dim3(32 * kRowWarps), 0, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, token_unsort_kernel<T, V>, a, nvec, nchunk);
}

template <typename T, int V>
static cudaError_t unsort_grad_as(const RowArgs &a, cudaStream_t stream) {
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)cap_grid(a.M, 64)), dim3(kGradThreads), 0, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, token_unsort_grad_kernel<T, V>, a, a.H / V);
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

// Calls F<T, V>(args, stream) for the element type and the widest access.
#define MOE_ROW_DISPATCH(F)                                                       \
    const int elem = dtype == MOE_DT_F32 ? 4 : 2;                                 \
    const int vb = vec_bytes(a, elem);                                            \
    if (dtype == MOE_DT_F32) return vb == 16 ? F<float, 4>(a, stream) : F<float, 1>(a, stream); \
    if (dtype == MOE_DT_F16)                                                      \
        return vb == 16 ? F<__half, 8>(a, stream)                                 \
                        : vb == 4 ? F<__half, 2>(a, stream) : F<__half, 1>(a, stream); \
    return vb == 16 ? F<__nv_bfloat16, 8>(a, stream)                              \
                    : vb == 4 ? F<__nv_bfloat16, 2>(a, stream) : F<__nv_bfloat16, 1>(a, stream);

cudaError_t launch_token_unsort(const void *rows, int64_t ldr, int dtype, int M, int k, int H,
                                const int32_t *route_row, const float *w, const void *residual,
                                int64_t ldres, void *out, int64_t ldo, cudaStream_t stream) {
    RowArgs a{};
    a.a = rows, a.res = residual, a.out = out, a.lda = ldr, a.ldres = ldres, a.ldout = ldo;
    a.route_row = route_row, a.w = w, a.M = M, a.k = k, a.H = H;
    MOE_ROW_DISPATCH(unsort_as)
}

cudaError_t launch_token_unsort_grad(const void *gout, int64_t ldo, const void *rows, int64_t ldr,
                                     int dtype, int M, int k, int H, const int32_t *route_row,
                                     const float *w, void *grows, int64_t ldg, float *gw,
                                     cudaStream_t stream) {
    RowArgs a{};
    a.a = gout, a.b = rows, a.out = grows, a.out2 = gw, a.lda = ldo, a.ldb = ldr, a.ldout = ldg;
    a.route_row = route_row, a.w = w, a.M = M, a.k = k, a.H = H;
    MOE_ROW_DISPATCH(unsort_grad_as)
}

}  // namespace moe
