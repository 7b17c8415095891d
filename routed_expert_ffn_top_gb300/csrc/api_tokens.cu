// api_tokens.cu -- C entry points (include/moe.h) of the token sort and of 4-bit block
// floating point: argument validation, tensor maps, and the 4-bit expert step.
#include <string.h>

#include "moe_internal.cuh"

using namespace moe;

static bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
static int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

static int dtype_bytes(int dtype) {
    return dtype == MOE_DT_F32 ? 4 : (dtype == MOE_DT_BF16 || dtype == MOE_DT_F16 ? 2 : 0);
}

static int check_routes(int M, int k) {
    if (M < 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (k > 32 || (int64_t)M * k >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// A matrix of `rows` rows of H elements, row pitch ld: its sizes, and its pointer's alignment
// to the element.
static int check_matrix(const void *p, int64_t ld, int H, int elem) {
    if (!p || ld < H || !aligned(p, elem)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// ------------------------------------------------------------------------------ token sort
extern "C" int moe_token_plan(const int32_t *topk_ids, int M, int k, int E, int32_t *offsets,
                              int32_t *row_route, int32_t *route_row, void *stream) {
    const int rc = check_routes(M, k);
    if (rc != MOE_OK) return rc;
    if (E <= 0) return MOE_ERR_INVALID_ARG;
    if (E > kPlanMaxExperts) return MOE_ERR_UNSUPPORTED;
    if (!offsets || !aligned(offsets, 4)) return MOE_ERR_INVALID_ARG;
    if (M > 0 && (!topk_ids || !row_route || !route_row || !aligned(topk_ids, 4) ||
                  !aligned(row_route, 4) || !aligned(route_row, 4)))
        return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_token_plan(topk_ids, M, k, E, offsets, row_route, route_row,
                                         static_cast<cudaStream_t>(stream)));
}

static int check_token_args(int dtype, int M, int k, int H, const int32_t *route_row) {
    const int rc = check_routes(M, k);
    if (rc != MOE_OK) return rc;
    if (dtype_bytes(dtype) == 0 || H <= 0) return MOE_ERR_INVALID_ARG;
    if (M > 0 && (!route_row || !aligned(route_row, 4))) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

extern "C" int moe_token_sort(const void *x, int64_t ldx, int dtype, int M, int k, int H,
                              const int32_t *route_row, void *rows, int64_t ldr, void *stream) {
    int rc = check_token_args(dtype, M, k, H, route_row);
    if (rc != MOE_OK) return rc;
    if (M == 0) return MOE_OK;
    const int elem = dtype_bytes(dtype);
    if ((rc = check_matrix(x, ldx, H, elem)) != MOE_OK) return rc;
    if ((rc = check_matrix(rows, ldr, H, elem)) != MOE_OK) return rc;
    return cuda_status(launch_token_sort(x, ldx, elem, M, k, H, route_row, rows, ldr,
                                         static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_token_sort_grad(const void *grad_rows, int64_t ldr, int dtype, int M, int k, int H,
                                   const int32_t *route_row, void *grad_x, int64_t ldx, void *stream) {
    return moe_token_unsort(grad_rows, ldr, dtype, M, k, H, route_row, nullptr, nullptr, 0, grad_x, ldx, stream);
}

extern "C" int moe_token_unsort(const void *rows, int64_t ldr, int dtype, int M, int k, int H,
                                const int32_t *route_row, const float *topk_weights,
                                const void *residual, int64_t ldres, void *out, int64_t ldo,
                                void *stream) {
    int rc = check_token_args(dtype, M, k, H, route_row);
    if (rc != MOE_OK) return rc;
    if (M == 0) return MOE_OK;
    const int elem = dtype_bytes(dtype);
    if ((rc = check_matrix(rows, ldr, H, elem)) != MOE_OK) return rc;
    if ((rc = check_matrix(out, ldo, H, elem)) != MOE_OK) return rc;
    if (residual && (rc = check_matrix(residual, ldres, H, elem)) != MOE_OK) return rc;
    if (topk_weights && !aligned(topk_weights, 4)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_token_unsort(rows, ldr, dtype, M, k, H, route_row, topk_weights, residual,
                                           residual ? ldres : 0, out, ldo, false, static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_token_unsort_grad(const void *grad_out, int64_t ldo, const void *rows, int64_t ldr,
                                     int dtype, int M, int k, int H, const int32_t *route_row,
                                     const float *topk_weights, void *grad_rows, int64_t ldg,
                                     float *grad_weights, void *stream) {
    int rc = check_token_args(dtype, M, k, H, route_row);
    if (rc != MOE_OK) return rc;
    if (M == 0) return MOE_OK;
    const int elem = dtype_bytes(dtype);
    if ((rc = check_matrix(grad_out, ldo, H, elem)) != MOE_OK) return rc;
    if ((rc = check_matrix(rows, ldr, H, elem)) != MOE_OK) return rc;
    if ((rc = check_matrix(grad_rows, ldg, H, elem)) != MOE_OK) return rc;
    if (!grad_weights || !aligned(grad_weights, 4) || (topk_weights && !aligned(topk_weights, 4)))
        return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_token_unsort_grad(grad_out, ldo, rows, ldr, dtype, M, k, H, route_row,
                                                topk_weights, grad_rows, ldg, grad_weights,
                                                static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------- 4-bit block floating point
// Columns of a quantised matrix: whole blocks, and rows short enough for 32-bit offsets.
static int check_cols(int cols) {
    if (cols <= 0) return MOE_ERR_INVALID_ARG;
    return cols % 32 != 0 || cols > (1 << 20) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

extern "C" int moe_microscale_pitch(int cols) { return check_cols(cols) == MOE_OK ? microscale_pitch(cols) : 0; }

extern "C" int moe_microscale_quantize(const void *x, int64_t ldx, int dtype, int64_t rows, int cols,
                                       const int32_t *route_row, int k, uint8_t *codes, uint8_t *scales,
                                       void *stream) {
    if (rows < 0 || dtype_bytes(dtype) == 0) return MOE_ERR_INVALID_ARG;
    int rc = check_cols(cols);
    if (rc != MOE_OK) return rc;
    if (rows >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
    if (route_row) {
        if (rows >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
        if ((rc = check_routes((int)rows, k)) != MOE_OK) return rc;
        if (!aligned(route_row, 4)) return MOE_ERR_INVALID_ARG;
    }
    if (rows == 0) return MOE_OK;
    if ((rc = check_matrix(x, ldx, cols, dtype_bytes(dtype))) != MOE_OK) return rc;
    if (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_microscale_quantize(x, ldx, dtype, rows, cols, route_row, route_row ? k : 1,
                                                  codes, scales, static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_microscale_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int cols,
                                         void *x, int64_t ldx, int dtype, void *stream) {
    if (rows < 0 || dtype_bytes(dtype) == 0) return MOE_ERR_INVALID_ARG;
    int rc = check_cols(cols);
    if (rc != MOE_OK) return rc;
    if (rows >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if ((rc = check_matrix(x, ldx, cols, dtype_bytes(dtype))) != MOE_OK) return rc;
    if (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_microscale_dequantize(codes, scales, rows, cols, x, ldx, dtype,
                                                    static_cast<cudaStream_t>(stream)));
}

// Sizes and pointers of a grouped product of rows [rows][K] and weights [E][N][K].
static int check_product(const uint8_t *x_codes, const uint8_t *x_scales, int64_t rows, const int32_t *offsets,
                         const uint8_t *w_codes, const uint8_t *w_scales, int E, int N, int K,
                         const void *workspace, size_t ws_bytes) {
    if (rows < 0 || E <= 0 || N <= 0) return MOE_ERR_INVALID_ARG;
    const int rc = check_cols(K);
    if (rc != MOE_OK) return rc;
    if (E > kMicroscaleMaxExperts || (int64_t)E * N >= ((int64_t)1 << 30) || rows >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
    if (!offsets && E != 1) return MOE_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) || (offsets && !aligned(offsets, 4))) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < MOE_MICROSCALE_STATUS_BYTES) return MOE_ERR_WORKSPACE;
    if (rows == 0) return MOE_OK;
    if (!x_codes || !x_scales || !w_codes || !w_scales) return MOE_ERR_INVALID_ARG;
    if (!aligned(x_codes, 16) || !aligned(x_scales, 16) || !aligned(w_codes, 16) || !aligned(w_scales, 16))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// The gated form's weights are seen as [chunk][gate/up][row]: one box takes a run of gate rows
// and the up rows beside it.  When K is not a whole number of copies the chunk dimension has
// one entry, a copy brings one chunk, and a row's bytes past its end read as zeros (a deeper
// box would zero-fill whole chunks past K, which costs as much as copying them).
static bool product_maps(MicroscaleMaps *tm, const uint8_t *x_codes, const uint8_t *x_scales, int64_t rows,
                         const uint8_t *w_codes, const uint8_t *w_scales, int E, int N, int K, bool gated,
                         void *y, int64_t ldy, int elem) {
    const MicroscaleTile t = microscale_tile(rows, E);
    const uint64_t row = (uint64_t)K / 2;
    const bool deep = K % (256 * t.chunks) == 0;
    const uint64_t inner = deep ? 128 : row, chunks = deep ? K / 256 : 1;
    const uint32_t depth = deep ? t.chunks : 1;
    const uint64_t halves = gated ? 2 : 1, wrows = (uint64_t)E * N - (gated ? N / 2 : 0);
    const uint64_t up = (uint64_t)(gated ? N / 2 : N);  // rows from gate to up
    const uint32_t bn = (uint32_t)(t.n / halves), m = (uint32_t)t.m, two = (uint32_t)halves;
    const CUtensorMapSwizzle sw128 = CU_TENSOR_MAP_SWIZZLE_128B;
    tm->deep = deep;
    tm->x_scales = x_scales;
    tm->w_scales = w_scales;
    const uint64_t ad[3] = {inner, (uint64_t)rows, chunks}, as[2] = {row, 128};
    const uint32_t ab[3] = {128, m, depth};
    const uint64_t bd[4] = {inner, wrows, halves, chunks}, bs[3] = {row, up * row, 128};
    const uint32_t bb[4] = {128, bn, two, depth};
    // y in bytes, boxes of 64 bytes x 32 rows, where its pointer and pitch allow tensor stores and
    // a row's bytes lie within their 32-bit signed coordinates
    tm->bulk = y && t.m == 128 && (reinterpret_cast<uintptr_t>(y) | (uint64_t)(ldy * elem)) % 16 == 0 &&
               (int64_t)N * elem <= INT32_MAX - 64;
    const uint64_t yd[2] = {(uint64_t)N * elem, (uint64_t)rows}, ys[1] = {(uint64_t)(ldy * elem)};
    const uint32_t yb[2] = {64, 32};
    if (!tm->bulk) memset(&tm->y, 0, sizeof tm->y);
    else if (!make_tmap_bytes(&tm->y, y, 2, yd, ys, yb, CU_TENSOR_MAP_SWIZZLE_64B)) return false;
    return make_tmap_bytes(&tm->x, x_codes, 3, ad, as, ab, sw128) &&
           make_tmap_bytes(&tm->w, w_codes, 4, bd, bs, bb, sw128);
}

static int product(const uint8_t *x_codes, const uint8_t *x_scales, int64_t rows, const int32_t *offsets,
                   const uint8_t *w_codes, const uint8_t *w_scales, int E, int N, int K, int dtype, void *y,
                   int64_t ldy, void *workspace, size_t ws_bytes, MicroscaleEarly early, void *stream) {
    int rc = check_product(x_codes, x_scales, rows, offsets, w_codes, w_scales, E, N, K, workspace, ws_bytes);
    if (rc != MOE_OK) return rc;
    if (dtype_bytes(dtype) == 0) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if ((rc = check_matrix(y, ldy, N, dtype_bytes(dtype))) != MOE_OK) return rc;
    MicroscaleMaps tm;
    if (!product_maps(&tm, x_codes, x_scales, rows, w_codes, w_scales, E, N, K, false, y, ldy, dtype_bytes(dtype))) return MOE_ERR_CUDA;
    return cuda_status(launch_microscale_gemm(tm, rows, offsets, E, N, K, dtype, y, ldy, nullptr, nullptr,
                                              early, static_cast<int32_t *>(workspace),
                                              static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_microscale_product(const uint8_t *x_codes, const uint8_t *x_scales, int64_t rows,
                                      const int32_t *offsets, const uint8_t *w_codes,
                                      const uint8_t *w_scales, int E, int N, int K, int dtype, void *y,
                                      int64_t ldy, void *workspace, size_t ws_bytes, void *stream) {
    return product(x_codes, x_scales, rows, offsets, w_codes, w_scales, E, N, K, dtype, y, ldy, workspace, ws_bytes,
                   MicroscaleEarly{}, stream);
}

static int gated_product(const uint8_t *x_codes, const uint8_t *x_scales, int64_t rows, const int32_t *offsets,
                         const uint8_t *w_codes, const uint8_t *w_scales, int E, int N, int K, uint8_t *codes,
                         uint8_t *scales, void *workspace, size_t ws_bytes, MicroscaleEarly early, void *stream) {
    int rc = check_product(x_codes, x_scales, rows, offsets, w_codes, w_scales, E, N, K, workspace, ws_bytes);
    if (rc != MOE_OK) return rc;
    if (N % 64 != 0) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16)) return MOE_ERR_INVALID_ARG;
    MicroscaleMaps tm;
    if (!product_maps(&tm, x_codes, x_scales, rows, w_codes, w_scales, E, N, K, true, nullptr, 0, 0)) return MOE_ERR_CUDA;
    return cuda_status(launch_microscale_gemm(tm, rows, offsets, E, N, K, MOE_DT_BF16, nullptr, 0, codes, scales,
                                              early, static_cast<int32_t *>(workspace),
                                              static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_microscale_gated_product(const uint8_t *x_codes, const uint8_t *x_scales, int64_t rows,
                                            const int32_t *offsets, const uint8_t *w_codes,
                                            const uint8_t *w_scales, int E, int N, int K, uint8_t *codes,
                                            uint8_t *scales, void *workspace, size_t ws_bytes, void *stream) {
    return gated_product(x_codes, x_scales, rows, offsets, w_codes, w_scales, E, N, K, codes, scales, workspace, ws_bytes,
                         MicroscaleEarly{}, stream);
}

// ----------------------------------------------------------------------- the expert step
struct MicroscaleWs {
    size_t offsets, row_route, route_row, x_codes, x_scales, p_codes, p_scales, y, total;
};

static MicroscaleWs microscale_ws(const moe_microscale_weights_t *w, int64_t R) {
    const int E = w->E, H = w->H, I = w->I;
    MicroscaleWs L;
    size_t off = MOE_MICROSCALE_STATUS_BYTES;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) / 256 * 256;
        return at;
    };
    L.offsets = take((size_t)(E + 1) * 4);
    L.row_route = take((size_t)R * 4);
    L.route_row = take((size_t)R * 4);
    L.x_codes = take((size_t)R * (H / 2));
    L.x_scales = take((size_t)R * microscale_pitch(H));
    L.p_codes = take((size_t)R * (I / 2));
    L.p_scales = take((size_t)R * microscale_pitch(I));
    L.y = take((size_t)R * H * dtype_bytes(w->y_dtype));
    L.total = off;
    return L;
}

static int check_microscale_weights(const moe_microscale_weights_t *w) {
    if (!w || w->H <= 0 || w->I <= 0 || w->E <= 0) return MOE_ERR_INVALID_ARG;
    if (w->y_dtype != MOE_DT_BF16 && w->y_dtype != MOE_DT_F32) return MOE_ERR_INVALID_ARG;
    if (check_cols(w->H) != MOE_OK || check_cols(w->I) != MOE_OK) return MOE_ERR_UNSUPPORTED;
    if (w->E > kMicroscaleMaxExperts || (int64_t)w->E * w->I * 2 >= ((int64_t)1 << 30) ||
        (int64_t)w->E * w->H >= ((int64_t)1 << 30))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

extern "C" size_t moe_microscale_workspace_bytes(const moe_microscale_weights_t *w, int M, int k) {
    if (check_microscale_weights(w) != MOE_OK || check_routes(M, k) != MOE_OK) return 0;
    return microscale_ws(w, (int64_t)M * k).total;
}

extern "C" int moe_microscale_ffn(const void *h, const moe_microscale_weights_t *w, int M, int k,
                                  const int32_t *topk_ids, const float *topk_weights, const void *residual,
                                  void *out, void *workspace, size_t ws_bytes, void *stream) {
    int rc = check_microscale_weights(w);
    if (rc != MOE_OK) return rc;
    if ((rc = check_routes(M, k)) != MOE_OK) return rc;
    if (M == 0) return MOE_OK;
    if (!h || !topk_ids || !topk_weights || !out || !workspace || !aligned(workspace, 256) ||
        !aligned(topk_ids, 4) || !aligned(topk_weights, 4) || !aligned(h, 16) || !aligned(out, 16) || (residual && !aligned(residual, 16)))
        return MOE_ERR_INVALID_ARG;
    for (const uint8_t *p : {w->gate_up_codes, w->gate_up_scales, w->down_codes, w->down_scales})
        if (!p || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    const int64_t R = (int64_t)M * k;
    const MicroscaleWs L = microscale_ws(w, R);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int32_t *offsets = reinterpret_cast<int32_t *>(ws + L.offsets);
    int32_t *route_row = reinterpret_cast<int32_t *>(ws + L.route_row);
    int32_t *row_route = reinterpret_cast<int32_t *>(ws + L.row_route);
    if (R <= kPlanQuantizeRoutes) {
        rc = cuda_status(launch_microscale_plan_quantize(static_cast<const __nv_bfloat16 *>(h), M, w->H, topk_ids, k, w->E,
                                                         offsets, row_route, route_row, ws + L.x_codes, ws + L.x_scales,
                                                         static_cast<cudaStream_t>(stream)));
    } else {
        rc = moe_token_plan(topk_ids, M, k, w->E, offsets, row_route, route_row, stream);
        if (rc != MOE_OK) return rc;
        rc = moe_microscale_quantize(h, w->H, MOE_DT_BF16, M, w->H, route_row, k, ws + L.x_codes, ws + L.x_scales, stream);
    }
    if (rc != MOE_OK) return rc;
    // The kernels of the step wait for the one ahead before they let the next begin.  So when the
    // gated product begins, the plan is complete, or where it is the kernel ahead, the caller's ids,
    // from which few routes' groups are counted; when the down product begins, so is the plan.
    // A product's first weights then arrive while the kernel ahead runs: one token's step 16.1 us
    // (waiting at the start 18.6), 21 tokens' 44.4 (47.9), 8192 tokens' 281 (287).
    const MicroscaleEarly planned{true, nullptr, 0}, count{true, topk_ids, (int)R};
    rc = gated_product(ws + L.x_codes, ws + L.x_scales, R, offsets, w->gate_up_codes, w->gate_up_scales, w->E, 2 * w->I,
                       w->H, ws + L.p_codes, ws + L.p_scales, workspace, ws_bytes,
                       R <= kPlanQuantizeRoutes ? count : planned, stream);
    if (rc != MOE_OK) return rc;
    // y in bf16 halves the largest transfer of the step at long prompts, for 2^-9 relative error on
    // each of k terms: without a residual 8192 tokens' result is 2.4e-3 off in the 2-norm instead of
    // 1.7e-3.  The caller chooses: with fp32 y they take 352 us for 278, one token 16.9 for 15.9.
    rc = product(ws + L.p_codes, ws + L.p_scales, R, offsets, w->down_codes, w->down_scales, w->E, w->H,
                 w->I, w->y_dtype, ws + L.y, w->H, workspace, ws_bytes, planned, stream);
    if (rc != MOE_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (w->y_dtype == MOE_DT_F32)
        return cuda_status(launch_token_unsort_f32(reinterpret_cast<float *>(ws + L.y), M, k, w->H, route_row, topk_weights,
                                                   static_cast<const __nv_bfloat16 *>(residual),
                                                   static_cast<__nv_bfloat16 *>(out), true, s));
    return cuda_status(launch_token_unsort(ws + L.y, w->H, MOE_DT_BF16, M, k, w->H, route_row, topk_weights, residual,
                                           residual ? w->H : 0, out, w->H, true, s));
}
