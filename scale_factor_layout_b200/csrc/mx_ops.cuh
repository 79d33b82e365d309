// mx_ops.cuh -- what the mixture-of-experts operators (sort, dispatch, combine,
// quantize, grouped product) share: argument limits, 16-byte vectors of a
// storage type, and the launch helper.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_device.cuh"
#include "mxscale.h"

// Defined in mx_rearrange.cu (C++ linkage, not part of the C ABI).
mx_status mx_record_cuda_error(cudaError_t e);
// Makes a context current in this thread if none is, and gives the SM count.
mx_status mx_device_sms(int *sms);

namespace mx {

constexpr int64_t kOpsMaxExtent = (1ll << 31) - (1ll << 14);

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t up_to(int64_t a, int64_t b) { return div_up(a, b) * b; }
// Strides are below 2^40 bytes: what a tensor map can hold, more than any memory has,
// and few enough that the host's arithmetic on them stays within 64 bits.
inline bool stride_fits(int64_t stride, int64_t element_bytes) { return stride < (1ll << 40) / element_bytes; }
// Whether rows of `cols` elements, `stride` apart, lie within `room` elements.
inline bool rows_fit(int64_t rows, int64_t stride, int64_t cols, int64_t room) {
    return rows < 1 || (cols <= room && (stride < 1 || rows - 1 <= (room - cols) / stride));
}
inline bool aligned_to(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A stream-ordered launch whose own return code is the result (the thread's
// pending CUDA error is neither read nor cleared).
template <typename... KArgs, typename... Args>
mx_status launch(void (*kernel)(KArgs...), int64_t grid, int block, int smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
    return e == cudaSuccess ? MX_OK : mx_record_cuda_error(e);
}

// Rows in groups, which is the first row behind the last group: the largest of the
// ends, as the group table's clamping has it (the table's cap, the number of rows,
// is left to the caller).  For whole warps.
__device__ __forceinline__ int rows_in_groups(const int *ends, int G) {
    const int lane = threadIdx.x & 31;
    const int e0 = lane < G ? __ldg(ends + lane) : 0, e1 = lane + 32 < G ? __ldg(ends + lane + 32) : 0;
    return max(0, __reduce_max_sync(0xffffffffu, max(e0, e1)));
}

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// N consecutive elements as one load or store moves them: 16 bytes, 8, 4, or one
// element, as rows are aligned.  They stay words until they are unpacked: arrays
// of 16-bit types are not always moved as a whole.
template <int bytes> struct RawOf;
template <> struct RawOf<16> { using Type = uint4; };
template <> struct RawOf<8> { using Type = uint2; };
template <> struct RawOf<4> { using Type = uint32_t; };
template <> struct RawOf<2> { using Type = uint16_t; };
template <typename T, int N> using Raw = typename RawOf<sizeof(T) * N>::Type;

template <typename T> __device__ __forceinline__ float2 two_floats(uint32_t w);
template <> __device__ __forceinline__ float2 two_floats<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 two_floats<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T> __device__ __forceinline__ uint32_t two_packed(float lo, float hi);
template <> __device__ __forceinline__ uint32_t two_packed<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t two_packed<__half>(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <typename T, int N>
__device__ __forceinline__ void unpack(const Raw<T, N> &r, float (&f)[N]) {
    if constexpr (N == 1 && sizeof(T) == 4) {
        f[0] = __uint_as_float(r);
    } else if constexpr (N == 1) {
        f[0] = two_floats<T>(r).x;
    } else if constexpr (N == 2 && sizeof(T) == 4) {
        f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y);
    } else if constexpr (N == 2) {
        const float2 a = two_floats<T>(r);
        f[0] = a.x, f[1] = a.y;
    } else if constexpr (N == 4 && sizeof(T) == 2) {
        const float2 a = two_floats<T>(r.x), b = two_floats<T>(r.y);
        f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    } else if constexpr (sizeof(T) == 4) {
        f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y), f[2] = __uint_as_float(r.z), f[3] = __uint_as_float(r.w);
    } else {
        const float2 a = two_floats<T>(r.x), b = two_floats<T>(r.y), c = two_floats<T>(r.z), d = two_floats<T>(r.w);
        f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y, f[4] = c.x, f[5] = c.y, f[6] = d.x, f[7] = d.y;
    }
}
template <typename T, int N>
__device__ __forceinline__ Raw<T, N> pack(const float (&f)[N]) {
    if constexpr (N == 1 && sizeof(T) == 4) {
        return __float_as_uint(f[0]);
    } else if constexpr (N == 1) {
        return (uint16_t)two_packed<T>(f[0], 0.f);
    } else if constexpr (N == 2 && sizeof(T) == 4) {
        return make_uint2(__float_as_uint(f[0]), __float_as_uint(f[1]));
    } else if constexpr (N == 2) {
        return two_packed<T>(f[0], f[1]);
    } else if constexpr (N == 4 && sizeof(T) == 2) {
        return make_uint2(two_packed<T>(f[0], f[1]), two_packed<T>(f[2], f[3]));
    } else if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
        return make_uint4(two_packed<T>(f[0], f[1]), two_packed<T>(f[2], f[3]), two_packed<T>(f[4], f[5]), two_packed<T>(f[6], f[7]));
    }
}

}  // namespace mx
