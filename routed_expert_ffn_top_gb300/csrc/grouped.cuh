// grouped.cuh -- launchers of the 16-bit grouped products and of the 8-bit checkpoints.
#pragma once

#include "moe_internal.cuh"

namespace moe {

constexpr int kGroupedMaxExperts = 1024;

// kWeights32: kWeights with an fp32 gradient.
enum class Grouped { kPlain, kGated, kGatedGrad, kWeights, kWeights32 };

// One grouped product (grouped_gemm.cu).  Channels: the columns of the result that lie on the
// MMA's M side (kPlain the output's, kGated and kGatedGrad I, kWeights the rows' columns K).
struct GroupedArgs {
    Grouped mode;
    int half;                 // operands, and 16-bit results, are f16, else bf16
    int transposed;           // kPlain: the weights are [E][channels][K]
    const int32_t *offsets;   // NULL: one group of all rows
    int64_t rows;
    int E, channels;
    int K;                    // summed length of a part (kWeights: rows are summed)
    int N;                    // kWeights: columns of the gradient
    int parts;                // kPlain: 1, or 2 for the sum of two products
    const void *x, *x2;       // rows [rows][K]: the M side's in kWeights
    int64_t ldx;
    const void *w, *w2;       // weights (kGated: gate, up); kWeights: grads [rows][N]
    int64_t ldw;              // kWeights: pitch of the grads
    void *out;                // kPlain y, kGated p, kGatedGrad grad of gate and up, kWeights the gradient
    int64_t ldo;
    int out_dtype;            // kPlain, kWeights: MOE_DT_*
    void *p;                  // kGatedGrad: p, contiguous, or NULL
    int code;                 // MOE_CODE_* of the checkpoint
    uint8_t *codes, *scales;  // checkpoint of gate and up side by side, or NULL (kGated)
    int32_t *status;
};
cudaError_t launch_grouped(const GroupedArgs &a, cudaStream_t stream);

// checkpoint.cu.  code: MOE_CODE_*.
cudaError_t launch_checkpoint_quantize(const void *x, int64_t ldx, int dtype, int64_t rows, int cols, int code,
                                       uint8_t *codes, uint8_t *scales, cudaStream_t stream);
cudaError_t launch_checkpoint_dequantize(const uint8_t *codes, const uint8_t *scales, int code, int64_t rows, int cols,
                                         const int32_t *route_row, int k, void *x, int64_t ldx, int dtype,
                                         cudaStream_t stream);

}  // namespace moe
