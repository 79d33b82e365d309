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

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// N consecutive elements moved by one load or store (16 bytes, or one element
// where rows do not start on 16-byte boundaries).
template <typename T, int N> struct alignas(sizeof(T) * N) Pack { T v[N]; };

}  // namespace mx
