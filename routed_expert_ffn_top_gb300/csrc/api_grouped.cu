// api_grouped.cu -- C entry points (include/moe.h) of the 16-bit grouped products and of the 8-bit
// checkpoints: argument validation.
#include "grouped.cuh"

using namespace moe;

static bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
static int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

static int dtype_bytes(int dtype) {
    return dtype == MOE_DT_F32 ? 4 : (dtype == MOE_DT_BF16 || dtype == MOE_DT_F16 ? 2 : 0);
}

static bool is_code(int code) { return code == MOE_CODE_E4M3 || code == MOE_CODE_INT8; }

// Columns of a 16-bit operand: tensor copies start and end on 16 bytes, and a row's bytes fit
// their coordinates.
static int check_width(int n) {
    if (n <= 0) return MOE_ERR_INVALID_ARG;
    return n % 8 != 0 || n > (1 << 20) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// What every grouped product checks first.
static int check_groups(int64_t rows, int dtype, const int32_t *offsets, int E, const void *workspace, size_t ws_bytes) {
    if (rows < 0 || E <= 0 || (dtype != MOE_DT_BF16 && dtype != MOE_DT_F16)) return MOE_ERR_INVALID_ARG;
    if (E > kGroupedMaxExperts || rows >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
    if (!offsets && E != 1) return MOE_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) || (offsets && !aligned(offsets, 4))) return MOE_ERR_INVALID_ARG;
    return ws_bytes < MOE_GROUPED_STATUS_BYTES ? MOE_ERR_WORKSPACE : MOE_OK;
}

// A 16-bit operand of `cols` columns.
static int check_operand(const void *p, int64_t ld, int64_t cols) {
    if (!p || ld < cols || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    return ld % 8 != 0 || ld >= ((int64_t)1 << 36) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

static GroupedArgs grouped_args(Grouped mode, const void *x, int64_t ldx, int64_t rows, int dtype, const int32_t *offsets,
                                int E, void *workspace) {
    GroupedArgs g{};
    g.mode = mode, g.x = x, g.ldx = ldx, g.rows = rows, g.half = dtype == MOE_DT_F16, g.offsets = offsets, g.E = E;
    g.parts = 1, g.out_dtype = dtype, g.status = static_cast<int32_t *>(workspace);
    return g;
}

extern "C" int moe_grouped_product(const void *x, int64_t ldx, int64_t rows, int dtype, const int32_t *offsets,
                                   const void *w, const void *w2, int transposed, int E, int N, int K, int y_dtype,
                                   void *y, int64_t ldy, void *workspace, size_t ws_bytes, void *stream) {
    int rc = check_groups(rows, dtype, offsets, E, workspace, ws_bytes);
    if (rc != MOE_OK || (rc = check_width(N)) != MOE_OK || (rc = check_width(K)) != MOE_OK) return rc;
    if (dtype_bytes(y_dtype) == 0) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if ((rc = check_operand(x, ldx, (int64_t)K * (w2 ? 2 : 1))) != MOE_OK) return rc;
    if (!w || !aligned(w, 16) || !aligned(w2, 16)) return MOE_ERR_INVALID_ARG;
    if (!y || ldy < N || !aligned(y, dtype_bytes(y_dtype))) return MOE_ERR_INVALID_ARG;
    GroupedArgs g = grouped_args(Grouped::kPlain, x, ldx, rows, dtype, offsets, E, workspace);
    g.channels = N, g.K = K, g.transposed = transposed != 0, g.w = w, g.w2 = w2, g.parts = w2 ? 2 : 1;
    g.x2 = static_cast<const uint16_t *>(x) + K;
    g.out = y, g.ldo = ldy, g.out_dtype = y_dtype;
    return cuda_status(launch_grouped(g, static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_grouped_gated_product(const void *x, int64_t ldx, int64_t rows, int dtype, const int32_t *offsets,
                                         const void *w_gate, const void *w_up, int E, int I, int H, void *p, int64_t ldp,
                                         int code, uint8_t *codes, uint8_t *scales, void *workspace, size_t ws_bytes,
                                         void *stream) {
    int rc = check_groups(rows, dtype, offsets, E, workspace, ws_bytes);
    if (rc != MOE_OK || (rc = check_width(I)) != MOE_OK || (rc = check_width(H)) != MOE_OK) return rc;
    if (I % 32 != 0 || I > (1 << 19)) return MOE_ERR_UNSUPPORTED;
    if ((codes == nullptr) != (scales == nullptr) || (codes && !is_code(code))) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if ((rc = check_operand(x, ldx, H)) != MOE_OK) return rc;
    if (!w_gate || !w_up || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(codes, 16) || !aligned(scales, 16))
        return MOE_ERR_INVALID_ARG;
    if (!p || ldp < I || !aligned(p, 2)) return MOE_ERR_INVALID_ARG;
    GroupedArgs g = grouped_args(Grouped::kGated, x, ldx, rows, dtype, offsets, E, workspace);
    g.channels = I, g.K = H, g.w = w_gate, g.w2 = w_up, g.out = p, g.ldo = ldp;
    g.code = code, g.codes = codes, g.scales = scales;
    return cuda_status(launch_grouped(g, static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_grouped_gated_product_grad(const void *grad_y, int64_t ldg, int64_t rows, int dtype,
                                              const int32_t *offsets, const void *w_down, int E, int I, int H, int code,
                                              const uint8_t *codes, const uint8_t *scales, void *grad_gate_up, void *p,
                                              void *workspace, size_t ws_bytes, void *stream) {
    int rc = check_groups(rows, dtype, offsets, E, workspace, ws_bytes);
    if (rc != MOE_OK || (rc = check_width(I)) != MOE_OK || (rc = check_width(H)) != MOE_OK) return rc;
    if (I % 32 != 0 || I > (1 << 19)) return MOE_ERR_UNSUPPORTED;
    if (!is_code(code)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if ((rc = check_operand(grad_y, ldg, H)) != MOE_OK) return rc;
    if (!w_down || !codes || !scales || !aligned(w_down, 16) || !aligned(codes, 16) || !aligned(scales, 16))
        return MOE_ERR_INVALID_ARG;
    if (!grad_gate_up || !aligned(grad_gate_up, 16) || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    GroupedArgs g = grouped_args(Grouped::kGatedGrad, grad_y, ldg, rows, dtype, offsets, E, workspace);
    g.channels = I, g.K = H, g.w = w_down, g.out = grad_gate_up, g.ldo = 2 * (int64_t)I, g.p = p;
    g.code = code, g.codes = const_cast<uint8_t *>(codes), g.scales = const_cast<uint8_t *>(scales);
    return cuda_status(launch_grouped(g, static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_grouped_weight_grad(const void *x, int64_t ldx, const void *grads, int64_t ldg, int64_t rows, int dtype,
                                       const int32_t *offsets, int E, int K, int N, int out_dtype, void *out,
                                       void *workspace, size_t ws_bytes, void *stream) {
    int rc = check_groups(rows, dtype, offsets, E, workspace, ws_bytes);
    if (rc != MOE_OK || (rc = check_width(N)) != MOE_OK || (rc = check_width(K)) != MOE_OK) return rc;
    if (dtype_bytes(out_dtype) == 0 || !out || !aligned(out, 16)) return MOE_ERR_INVALID_ARG;
    // tiles are counted in 32 bits
    if ((int64_t)E * ((N + 255) / 256) * ((K + 255) / 256) >= ((int64_t)1 << 30)) return MOE_ERR_UNSUPPORTED;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) return cuda_status(cudaMemsetAsync(out, 0, (size_t)E * K * N * dtype_bytes(out_dtype), s));
    if ((rc = check_operand(x, ldx, K)) != MOE_OK || (rc = check_operand(grads, ldg, N)) != MOE_OK) return rc;
    GroupedArgs g = grouped_args(Grouped::kWeights, x, ldx, rows, dtype, offsets, E, workspace);
    g.channels = K, g.N = N, g.w = grads, g.ldw = ldg, g.out = out, g.out_dtype = out_dtype;
    return cuda_status(launch_grouped(g, s));
}

// ------------------------------------------------------------------------ 8-bit checkpoints
static int check_cols(int cols) {
    if (cols <= 0) return MOE_ERR_INVALID_ARG;
    return cols % 32 != 0 || cols > (1 << 20) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

extern "C" int moe_checkpoint_pitch(int cols) { return check_cols(cols) == MOE_OK ? microscale_pitch(cols) : 0; }

extern "C" int moe_checkpoint_quantize(const void *x, int64_t ldx, int dtype, int64_t rows, int cols, int code,
                                       uint8_t *codes, uint8_t *scales, void *stream) {
    if (rows < 0 || dtype_bytes(dtype) == 0 || !is_code(code)) return MOE_ERR_INVALID_ARG;
    const int rc = check_cols(cols);
    if (rc != MOE_OK) return rc;
    if (rows >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!x || ldx < cols || !aligned(x, dtype_bytes(dtype))) return MOE_ERR_INVALID_ARG;
    if (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_checkpoint_quantize(x, ldx, dtype, rows, cols, code, codes, scales,
                                                  static_cast<cudaStream_t>(stream)));
}

extern "C" int moe_checkpoint_dequantize(const uint8_t *codes, const uint8_t *scales, int code, int64_t rows, int cols,
                                         const int32_t *route_row, int k, void *x, int64_t ldx, int dtype, void *stream) {
    if (rows < 0 || dtype_bytes(dtype) == 0 || !is_code(code)) return MOE_ERR_INVALID_ARG;
    const int rc = check_cols(cols);
    if (rc != MOE_OK) return rc;
    if (rows >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
    if (route_row) {
        if (k <= 0 || !aligned(route_row, 4)) return MOE_ERR_INVALID_ARG;
        if (k > 32 || rows * k >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
    }
    if (rows == 0) return MOE_OK;
    if (!x || ldx < cols || !aligned(x, dtype_bytes(dtype))) return MOE_ERR_INVALID_ARG;
    if (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_checkpoint_dequantize(codes, scales, code, rows, cols, route_row, route_row ? k : 1, x, ldx,
                                                    dtype, static_cast<cudaStream_t>(stream)));
}
