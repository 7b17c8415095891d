// microscale.cu -- 4-bit block floating point (the OCP Microscaling Formats Specification's
// MXFP4): quantisation of rows and the way back.
//
// A block is 32 consecutive values of a row.  Its scale is a power of two 2^X held as the
// byte X + 127, with X = clamp(floor(log2 max|x|) - 2, -127, 127) (2 is the exponent of the
// largest code, 6 = 1.5 * 2^2); a value's code is x / 2^X rounded to the nearest of
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign, ties to the even code, saturating at 6.  Division
// by 2^X is exact, so each value is rounded once.  A block without a nonzero value has scale
// byte 0; a block with an infinity or a NaN has scale byte 255, which makes all its values
// NaN, and codes 0.
//
// Codes are packed two to a byte, the even column in the low half: [rows][cols / 2].  Scale
// rows are padded to a multiple of 16 bytes, [rows][pitch] (the tensor-map rule on row
// pitches), and the padding is written as 0.
#include "microscale.cuh"

namespace moe {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

// Sixteen consecutive elements by accesses of kBytes (32, 16, or the element's).
template <typename T, int kBytes>
__device__ __forceinline__ void load16(const T *p, float (&v)[16]) {
    if constexpr (kBytes >= 16) {
        alignas(32) uint32_t u[4 * sizeof(T)];
        constexpr int words = kBytes / 4;
#pragma unroll
        for (int i = 0; i < (int)(4 * sizeof(T)); i += words) {
            const uint32_t *q = reinterpret_cast<const uint32_t *>(p) + i;
            if constexpr (kBytes == 32)
                asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                             : "=r"(u[i]), "=r"(u[i + 1]), "=r"(u[i + 2]), "=r"(u[i + 3]), "=r"(u[i + 4]),
                               "=r"(u[i + 5]), "=r"(u[i + 6]), "=r"(u[i + 7])
                             : "l"(q));
            else
                *reinterpret_cast<uint4 *>(&u[i]) = *reinterpret_cast<const uint4 *>(q);
        }
        const T *t = reinterpret_cast<const T *>(u);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = to_f32(t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = to_f32(p[i]);
    }
}

struct QuantArgs {
    const void *x;
    int64_t ldx;
    int64_t rows;
    int cols, pitch, k;
    const int32_t *route_row;  // NULL: row m goes to row m; else to the rows of its k routes
    uint8_t *codes, *scales;
};

// A unit is 512 columns of one row, one warp: lane l takes columns 16 l to 16 l + 15, two lanes
// share a block.  512 columns are 16 scale bytes, one store.  With route_row a token is
// quantised once and stored k times (tail rows of dropped routes as zeros).
// Memory bound: elem + 1/2 + 1/32 bytes a value.  128 x 1536 rows of 2048 bf16: 156 us, 6.5 TB/s,
// 0.96 of the copy rate; 8192 tokens into 65,536 sorted rows: 19.6 us, 0.79.
// kRouted: row_l holds in lane j < k the route_row entry of slot j; else the unit goes to row m.
template <typename T, int kBytes, bool kRouted>
__device__ __forceinline__ void quantize_unit(const QuantArgs &a, int64_t m, int c0, int row_l) {
    const int lane = threadIdx.x & 31;
    const bool in = c0 + lane * 16 < a.cols;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    if (in) load16<T, kBytes>(static_cast<const T *>(a.x) + m * a.ldx + c0 + lane * 16, v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
        top = b > top ? b : top;
    }
    const uint32_t other = __shfl_xor_sync(0xffffffffu, top, 1);
    const uint32_t byte = microscale_byte(other > top ? other : top);
    const float inv = microscale_inverse(byte);
    float f[2][8];
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i / 8][i % 8] = v[i] * inv;
    uint2 code = {fp4x8(f[0]), fp4x8(f[1])};
    if (byte == 255u) code = {0u, 0u};
    // the warp's 16 scale bytes, block b's in lane 2 b: pairs, then fours, then all in lane 0
    uint32_t s4 = byte | __shfl_down_sync(0xffffffffu, byte, 2) << 8;
    s4 |= __shfl_down_sync(0xffffffffu, s4, 4) << 16;
    uint4 sc;
    sc.x = s4;
    sc.y = __shfl_down_sync(0xffffffffu, s4, 8);
    sc.z = __shfl_down_sync(0xffffffffu, s4, 16);
    sc.w = __shfl_down_sync(0xffffffffu, s4, 24);
    uint8_t *codes = a.codes + (c0 + lane * 16) / 2, *scales = a.scales + c0 / 32;
    const uint32_t half = (uint32_t)a.cols / 2, pitch = (uint32_t)a.pitch;
    if constexpr (!kRouted) {
        if (in) *reinterpret_cast<uint2 *>(codes + (uint64_t)m * half) = code;
        if (lane == 0) *reinterpret_cast<uint4 *>(scales + (uint64_t)m * pitch) = sc;
    } else {
        const uint32_t R = (uint32_t)a.rows * (uint32_t)a.k;  // below 2^24
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) {
            const int row = __shfl_sync(0xffffffffu, row_l, j);
            const bool live = row >= 0;
            const uint32_t at = (uint32_t)(live ? row : ~row);
            if (at >= R) continue;
            if (in) *reinterpret_cast<uint2 *>(codes + (uint64_t)at * half) = live ? code : uint2{0u, 0u};
            if (lane == 0) *reinterpret_cast<uint4 *>(scales + (uint64_t)at * pitch) = live ? sc : uint4{0, 0, 0, 0};
        }
    }
}

template <typename T, int kBytes, bool kRouted>
__global__ void __launch_bounds__(256) microscale_quantize_kernel(const QuantArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t stride = (int64_t)gridDim.x * 8;
    for (int64_t m = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); m < a.rows; m += stride) {
        const int row_l = kRouted && lane < a.k ? a.route_row[m * a.k + lane] : 0;
        quantize_unit<T, kBytes, kRouted>(a, m, blockIdx.y * 512, row_l);
    }
}

// The token plan and the quantisation into sorted rows of few routes in one launch: every CTA
// ranks the routes by comparing each with all others (the plan's order: expert, then route;
// dropped ones last), the first one writes the plan.
__global__ void __launch_bounds__(kPlanQuantizeRoutes)
microscale_plan_quantize_kernel(const QuantArgs a, const int32_t *ids, int E, int32_t *offsets,
                                int32_t *row_route, int32_t *route_row) {
    __shared__ int4 key4[kPlanQuantizeRoutes / 4];
    __shared__ int row[kPlanQuantizeRoutes];
    int *key = reinterpret_cast<int *>(key4);
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, r = threadIdx.x, R = (int)a.rows * a.k;
    const int id = r < R ? ids[r] : 0;
    const int mine = r < R ? ((uint32_t)id < (uint32_t)E ? id : E) : E + 1;
    key[r] = mine;
    __syncthreads();
    int at = 0;
    for (int i = 0; i < (R + 3) / 4; ++i) {
        const int4 q = key4[i];
        at += (q.x < mine || (q.x == mine && 4 * i < r)) + (q.y < mine || (q.y == mine && 4 * i + 1 < r)) +
              (q.z < mine || (q.z == mine && 4 * i + 2 < r)) + (q.w < mine || (q.w == mine && 4 * i + 3 < r));
    }
    row[r] = mine < E ? at : ~at;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        if (r < R) {
            route_row[r] = mine < E ? at : ~at;
            row_route[at] = mine < E ? r : -1;
        }
        for (int e = r; e <= E; e += kPlanQuantizeRoutes) {
            int n = 0;
            for (int i = 0; i < (R + 3) / 4; ++i) {
                const int4 q = key4[i];
                n += (q.x < e) + (q.y < e) + (q.z < e) + (q.w < e);
            }
            offsets[e] = n;
        }
    }
    __syncthreads();
    const int64_t stride = (int64_t)gridDim.x * (kPlanQuantizeRoutes / 32);
    for (int64_t m = (int64_t)blockIdx.x * (kPlanQuantizeRoutes / 32) + (threadIdx.x >> 5); m < a.rows; m += stride)
        quantize_unit<__nv_bfloat16, 16, true>(a, m, blockIdx.y * 512, lane < a.k ? row[m * a.k + lane] : 0);
}

struct DequantArgs {
    const uint8_t *codes, *scales;
    int64_t rows;
    int cols, pitch;
    void *x;
    int64_t ldx;
};

// Eight codes to four bf16 pairs: the two bytes of a magnitude's bf16 come from two eight-entry
// byte tables indexed by the code, the sign bits are moved in.
__device__ __forceinline__ void decode_bf16(uint32_t code, uint32_t (&v)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t c = code >> (16 * h), sel = c & 0x7777u;
        const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, sel);
        const uint32_t lo = __byte_perm(0xc0800000u, 0xc0804000u, sel);
        v[2 * h] = __byte_perm(lo, hi, 0x5140) | ((c & 0x8u) << 12) | ((c & 0x80u) << 24);
        v[2 * h + 1] = __byte_perm(lo, hi, 0x7362) | ((c & 0x800u) << 4) | ((c & 0x8000u) << 16);
    }
}

// Eight values of a block: the products with 2^X are exact in bf16 and fp32.
__device__ __forceinline__ void decode8(uint32_t code, uint32_t byte, __nv_bfloat16 (&o)[8]) {
    uint32_t v[4];
    decode_bf16(code, v);
    const uint32_t s = byte == 255u ? 0x7fffu : (byte == 0u ? 0x0040u : byte << 7);
    const uint32_t ss = s | (s << 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<__nv_bfloat162 *>(&o[2 * i]) = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&v[i]),
                                                                 *reinterpret_cast<const __nv_bfloat162 *>(&ss));
}
__device__ __forceinline__ void decode8(uint32_t code, uint32_t byte, float (&o)[8]) {
    uint32_t v[4];
    decode_bf16(code, v);
    const float s = microscale_value(byte);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = bf16_lo(v[i]) * s;
        o[2 * i + 1] = bf16_hi(v[i]) * s;
    }
}
__device__ __forceinline__ void decode8(uint32_t code, uint32_t byte, __half (&o)[8]) {
    float f[8];
    decode8(code, byte, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __float2half_rn(f[i]);
}

// A unit is 512 columns of one row, as above.  A code's value times 2^X is exact in fp32 and
// in bf16; fp16 rounds it (to infinity past its range).  128 x 1536 rows of 2048 to bf16: 160 us,
// 0.94 of the copy rate (269 with a code's value worked out bit by bit).
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) microscale_dequantize_kernel(const DequantArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, c0 = blockIdx.y * 512 + lane * 8;
    const int64_t stride = (int64_t)gridDim.x * 8;
    for (int64_t m = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); m < a.rows; m += stride) {
        uint32_t code[2], byte[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + 256 * h;
            code[h] = c < a.cols ? *reinterpret_cast<const uint32_t *>(a.codes + m * (a.cols / 2) + c / 2) : 0u;
            byte[h] = c < a.cols ? a.scales[m * a.pitch + c / 32] : 0u;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + 256 * h;
            if (c >= a.cols) continue;
            alignas(16) T o[8];
            decode8(code[h], byte[h], o);
            T *dst = static_cast<T *>(a.x) + m * a.ldx + c;
            if constexpr (kVec) {
                constexpr int n = 16 / sizeof(T);
#pragma unroll
                for (int i = 0; i < 8; i += n)
                    *reinterpret_cast<uint4 *>(dst + i) = *reinterpret_cast<const uint4 *>(&o[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[i] = o[i];
            }
        }
    }
}

// Grid: rows along x, 512-column chunks along y; up to 64 CTAs an SM in all.
static dim3 rows_by_chunks(int64_t rows, int cols) {
    const int64_t nchunk = (cols + 511) / 512, n = (rows + 7) / 8, most = (int64_t)num_sms() * 64 / nchunk + 1;
    return dim3((unsigned)(n < most ? n : most), (unsigned)nchunk);
}

template <typename T, bool kRouted>
static cudaError_t quantize_as(const QuantArgs &a, cudaStream_t stream) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(a.x) | (uint64_t)(a.ldx * sizeof(T));
    const auto fn = bits % 32 == 0   ? microscale_quantize_kernel<T, 32, kRouted>
                    : bits % 16 == 0 ? microscale_quantize_kernel<T, 16, kRouted>
                                     : microscale_quantize_kernel<T, (int)sizeof(T), kRouted>;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(rows_by_chunks(a.rows, a.cols), dim3(256), 0, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, fn, a);
}

template <typename T>
static cudaError_t dequantize_as(const DequantArgs &a, cudaStream_t stream) {
    const bool vec = (reinterpret_cast<uintptr_t>(a.x) | (uint64_t)(a.ldx * sizeof(T))) % 16 == 0;
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(rows_by_chunks(a.rows, a.cols), dim3(256), 0, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, vec ? microscale_dequantize_kernel<T, true> : microscale_dequantize_kernel<T, false>, a);
}

cudaError_t launch_microscale_quantize(const void *x, int64_t ldx, int dtype, int64_t rows, int cols,
                                       const int32_t *route_row, int k, uint8_t *codes, uint8_t *scales,
                                       cudaStream_t stream) {
    const QuantArgs a{x, ldx, rows, cols, microscale_pitch(cols), k, route_row, codes, scales};
    if (dtype == MOE_DT_F32) return route_row ? quantize_as<float, true>(a, stream) : quantize_as<float, false>(a, stream);
    if (dtype == MOE_DT_F16) return route_row ? quantize_as<__half, true>(a, stream) : quantize_as<__half, false>(a, stream);
    return route_row ? quantize_as<__nv_bfloat16, true>(a, stream) : quantize_as<__nv_bfloat16, false>(a, stream);
}

cudaError_t launch_microscale_plan_quantize(const __nv_bfloat16 *x, int M, int cols, const int32_t *ids, int k,
                                            int E, int32_t *offsets, int32_t *row_route, int32_t *route_row,
                                            uint8_t *codes, uint8_t *scales, cudaStream_t stream) {
    const QuantArgs a{x, cols, M, cols, microscale_pitch(cols), k, route_row, codes, scales};
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = launch_config(rows_by_chunks(M, cols), dim3(kPlanQuantizeRoutes), 0, stream, attrs, 0);
    return cudaLaunchKernelEx(&cfg, microscale_plan_quantize_kernel, a, ids, E, offsets, row_route, route_row);
}

cudaError_t launch_microscale_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                         int cols, void *x, int64_t ldx, int dtype, cudaStream_t stream) {
    const DequantArgs a{codes, scales, rows, cols, microscale_pitch(cols), x, ldx};
    if (dtype == MOE_DT_F32) return dequantize_as<float>(a, stream);
    if (dtype == MOE_DT_F16) return dequantize_as<__half>(a, stream);
    return dequantize_as<__nv_bfloat16>(a, stream);
}

}  // namespace moe
