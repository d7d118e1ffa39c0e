// Device helpers of the activation-side kernels: element types, the 8-bit block rule, and the
// launch with programmatic stream serialization. Internal; everything in an anonymous namespace.
//
// Order on the stream. Every kernel here waits for the kernel before it to complete before its
// first access to memory (griddepcontrol.wait), and none lets the next kernel on the stream
// start early, except a call's own second kernel: so a call is ordered like an ordinary launch,
// also between the calls of a zero_overlap_begin/end region.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "zero_act.h"
#include "zero_device.cuh"

namespace zk {
namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }

// v as it reads back from memory in type T.
template <typename T>
__device__ __forceinline__ float round_to(float v) { return to_f(from_f<T>(v)); }

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The scale of a block from the largest |x| as binary32 bits (they order like the values; an inf
// or NaN is at or above 0x7f800000 and makes the scale NaN).
__device__ __forceinline__ float q8_scale(uint32_t amax) {
    return amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                               : __fdiv_rn(__uint_as_float(amax), 127.0f);
}

// Code byte of x. A scale of 0 or NaN gives q = 0. The quotient of a subnormal scale can pass
// 127 (the scale itself was rounded): clamped.
__device__ __forceinline__ uint32_t q8_code(float x, float scale) {
    if (!(scale > 0.0f)) return 128u;
    const int q = __float2int_rn(__fdiv_rn(x, scale));
    return (uint32_t)(min(max(q, -127), 127) + 128);
}

__device__ __forceinline__ float q8_value(uint32_t byte, float scale) {
    return __fmul_rn((float)((int)byte - 128), scale);
}

__device__ __forceinline__ const float* ckpt_scales(const uint8_t* row, const CkptShape& s) {
    return reinterpret_cast<const float*>(row + s.code_bytes);
}

__device__ __forceinline__ void grid_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_launch_next() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename K, typename... A>
cudaError_t launch_act(K kernel, dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                       A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    count_launch();
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace
}  // namespace zk
