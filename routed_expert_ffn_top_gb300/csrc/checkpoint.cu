// checkpoint.cu -- activations in 8 bits: quantisation of rows and the way back, into token order
// or into the sorted order of a token plan.
//
// A block is 32 consecutive values of a row.  Its scale is a power of two 2^X held as the byte
// X + 127, with X the smallest integer from -127 up with max|x| <= Q 2^X; Q is the largest code,
// 448 (E4M3) or 127 (int8).  A value's code is x / 2^X rounded to the nearest code, ties to even.
// Division by 2^X is exact and no code saturates, so a value x is off by at most half a step of its
// code: 2^-4 |x| or, below 2^-6 2^X, 2^-10 2^X in E4M3; 2^X / 2 in int8, which is max / 127 at most where
// X > -127.  (A scale of any other value would round the quotient first, and a code next to a border
// would depend on how.)
// A block without a nonzero value has scale byte 0; a block with an infinity or a NaN has scale
// byte 255, which makes all its values NaN, and codes 0.  int8 keeps no sign of zero.
//
// codes [rows][cols], scales [rows][pitch] with pitch = cols / 32 rounded up to 16, padding 0.
#include "checkpoint.cuh"
#include "grouped.cuh"
#include "row_io.cuh"

namespace moe {

struct EightArgs {
    const void *x;
    void *out;
    int64_t ld;  // row pitch of x, or of the values written
    int64_t rows;
    int cols, pitch, k;
    const int32_t *route_row;  // NULL: row m goes to row m; else to the rows of its k routes
    uint8_t *codes, *scales;
};

// A unit is 512 columns of one row, one warp: lane l takes columns 16 l to 16 l + 15, two lanes
// share a block; 512 columns are 16 scale bytes, one store.  Memory bound: elem + 1 + 1/32 bytes
// a value: 8192 x 2048 bf16 in 10 us, 5.1 TB/s.
template <typename T, int kBytes, bool kInt8>
__global__ void __launch_bounds__(256) eight_quantize_kernel(const EightArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, c0 = blockIdx.y * 512, c = c0 + lane * 16;
    const bool in = c < a.cols;
    const int64_t stride = (int64_t)gridDim.x * 8;
    for (int64_t m = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); m < a.rows; m += stride) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.0f;
        if (in) load16<T, kBytes>(static_cast<const T *>(a.x) + m * a.ld + c, v);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
            top = b > top ? b : top;
        }
        const uint32_t other = __shfl_xor_sync(0xffffffffu, top, 1);
        const uint32_t byte = eight_byte<kInt8>(other > top ? other : top);
        const uint4 code = eight_codes<kInt8>(v, byte);
        // the warp's 16 scale bytes, block b's in lane 2 b: pairs, then fours, then all in lane 0
        uint32_t s4 = byte | __shfl_down_sync(0xffffffffu, byte, 2) << 8;
        s4 |= __shfl_down_sync(0xffffffffu, s4, 4) << 16;
        uint4 sc;
        sc.x = s4;
        sc.y = __shfl_down_sync(0xffffffffu, s4, 8);
        sc.z = __shfl_down_sync(0xffffffffu, s4, 16);
        sc.w = __shfl_down_sync(0xffffffffu, s4, 24);
        if (in) *reinterpret_cast<uint4 *>(a.codes + m * a.cols + c) = code;
        if (lane == 0) *reinterpret_cast<uint4 *>(a.scales + m * a.pitch + c0 / 32) = sc;
    }
}

// Sixteen values of T to dst by stores of kBytes (32, 16, or the element's).
template <typename T, int kBytes>
__device__ __forceinline__ void store16(T *dst, const T (&o)[16]) {
    const uint32_t *u = reinterpret_cast<const uint32_t *>(&o[0]);
    if constexpr (kBytes == 32) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) * 4; i += 8) st_global_32(reinterpret_cast<uint32_t *>(dst) + i, u + i);
    } else if constexpr (kBytes == 16) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) * 4; i += 4)
            *reinterpret_cast<uint4 *>(reinterpret_cast<uint32_t *>(dst) + i) = make_uint4(u[i], u[i + 1], u[i + 2], u[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[i] = o[i];
    }
}

// A unit as above.  With route_row a token's codes are read once and its values stored to the rows
// of its k routes (zeros to a dropped route's row).  A value is exact in fp32, and in bf16 from 2^-126 up;
// fp16 rounds it, to infinity past its range.  Memory bound: 8192 tokens of 2048 into 65,536 rows in 45
// us, 6.3 TB/s, 0.93 of the copy rate.
template <typename T, int kBytes, bool kInt8, bool kRouted>
__global__ void __launch_bounds__(256) eight_dequantize_kernel(const EightArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, c = blockIdx.y * 512 + lane * 16;
    const bool in = c < a.cols;
    const int64_t stride = (int64_t)gridDim.x * 8;
    for (int64_t m = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); m < a.rows; m += stride) {
        const int row_l = kRouted && lane < a.k ? a.route_row[m * a.k + lane] : 0;
        uint4 code{0, 0, 0, 0};
        uint32_t byte = 0;
        if (in) {
            code = *reinterpret_cast<const uint4 *>(a.codes + m * a.cols + c);
            byte = a.scales[m * a.pitch + c / 32];
        }
        float v[16];
        eight_values<kInt8>(code, byte, v);
        alignas(32) T o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) put_f32(&o[i], v[i]);
        T *out = static_cast<T *>(a.out) + c;
        if constexpr (!kRouted) {
            if (in) store16<T, kBytes>(out + m * a.ld, o);
        } else {
            const uint32_t R = (uint32_t)a.rows * (uint32_t)a.k;  // below 2^24
            alignas(32) T zero[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) put_f32(&zero[i], 0.0f);
#pragma unroll 4
            for (int j = 0; j < a.k; ++j) {
                const int row = __shfl_sync(0xffffffffu, row_l, j);
                const uint32_t at = (uint32_t)(row >= 0 ? row : ~row);
                if (at >= R || !in) continue;
                if (row >= 0) store16<T, kBytes>(out + at * a.ld, o);
                else store16<T, kBytes>(out + at * a.ld, zero);
            }
        }
    }
}

// Grid: rows along x, 512-column chunks along y; up to 64 CTAs an SM in all.
static dim3 rows_by_chunks(int64_t rows, int cols) {
    const int64_t nchunk = (cols + 511) / 512, n = (rows + 7) / 8, most = (int64_t)num_sms() * 64 / nchunk + 1;
    return dim3((unsigned)(n < most ? n : most), (unsigned)nchunk);
}

template <typename T, bool kInt8>
static cudaError_t quantize_as(const EightArgs &a, cudaStream_t stream) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(a.x) | (uint64_t)(a.ld * sizeof(T));
    const auto fn = bits % 32 == 0   ? eight_quantize_kernel<T, 32, kInt8>
                    : bits % 16 == 0 ? eight_quantize_kernel<T, 16, kInt8>
                                     : eight_quantize_kernel<T, (int)sizeof(T), kInt8>;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(rows_by_chunks(a.rows, a.cols), dim3(256), 0, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, fn, a);
}

template <typename T, bool kInt8, bool kRouted>
static cudaError_t dequantize_routed(const EightArgs &a, cudaStream_t stream) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(a.out) | (uint64_t)(a.ld * sizeof(T));
    const auto fn = bits % 32 == 0   ? eight_dequantize_kernel<T, 32, kInt8, kRouted>
                    : bits % 16 == 0 ? eight_dequantize_kernel<T, 16, kInt8, kRouted>
                                     : eight_dequantize_kernel<T, (int)sizeof(T), kInt8, kRouted>;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(rows_by_chunks(a.rows, a.cols), dim3(256), 0, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, fn, a);
}

template <typename T, bool kInt8>
static cudaError_t dequantize_as(const EightArgs &a, cudaStream_t stream) {
    return a.route_row ? dequantize_routed<T, kInt8, true>(a, stream) : dequantize_routed<T, kInt8, false>(a, stream);
}

cudaError_t launch_checkpoint_quantize(const void *x, int64_t ldx, int dtype, int64_t rows, int cols, int code,
                                       uint8_t *codes, uint8_t *scales, cudaStream_t stream) {
    const EightArgs a{x, nullptr, ldx, rows, cols, microscale_pitch(cols), 1, nullptr, codes, scales};
    const bool i8 = code == MOE_CODE_INT8;
    if (dtype == MOE_DT_F32) return i8 ? quantize_as<float, true>(a, stream) : quantize_as<float, false>(a, stream);
    if (dtype == MOE_DT_F16) return i8 ? quantize_as<__half, true>(a, stream) : quantize_as<__half, false>(a, stream);
    return i8 ? quantize_as<__nv_bfloat16, true>(a, stream) : quantize_as<__nv_bfloat16, false>(a, stream);
}

cudaError_t launch_checkpoint_dequantize(const uint8_t *codes, const uint8_t *scales, int code, int64_t rows, int cols,
                                         const int32_t *route_row, int k, void *x, int64_t ldx, int dtype,
                                         cudaStream_t stream) {
    const EightArgs a{nullptr, x, ldx, rows, cols, microscale_pitch(cols), k, route_row, const_cast<uint8_t *>(codes),
                      const_cast<uint8_t *>(scales)};
    const bool i8 = code == MOE_CODE_INT8;
    if (dtype == MOE_DT_F32) return i8 ? dequantize_as<float, true>(a, stream) : dequantize_as<float, false>(a, stream);
    if (dtype == MOE_DT_F16) return i8 ? dequantize_as<__half, true>(a, stream) : dequantize_as<__half, false>(a, stream);
    return i8 ? dequantize_as<__nv_bfloat16, true>(a, stream) : dequantize_as<__nv_bfloat16, false>(a, stream);
}

}  // namespace moe
