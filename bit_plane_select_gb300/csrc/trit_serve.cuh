// Device helpers of the decode step between the products: the batch's
// geometry, the 16-bit types and the launch with programmatic stream
// serialisation.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "trit_internal.cuh"

namespace trit {

__device__ __forceinline__ void raise_flag(uint32_t *err, uint32_t bit) {
    if ((*reinterpret_cast<volatile uint32_t *>(err) & bit) == 0) atomicOr(err, bit);
}

// The number of valid new tokens of sequence b, clamped to [0, T]; with an `err`, a
// number outside that range is flagged there.
__device__ __forceinline__ int batch_new(const trit_kv_batch &B, int b, uint32_t *err = nullptr) {
    const int n = B.new_lens ? B.new_lens[b] : B.T;
    if (n >= 0 && n <= B.T) return n;
    if (err) raise_flag(err, TRIT_ERR_INDEX);
    return n < 0 ? 0 : B.T;
}

// Two fp32 values as a pair of 16-bit ones, x in the low half, rounded to nearest even.
template <typename T>
__device__ __forceinline__ uint32_t pack16(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float x, float y) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
    return d;
}
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float x, float y) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
    return d;
}
template <typename T>
__device__ __forceinline__ float2 unpack16(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack16<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack16<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// Launches kernel with programmatic stream serialisation: its CTAs may start
// while the preceding grid drains; the kernel waits (griddepcontrol.wait)
// before it touches memory that grid may write or read.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;"); }

}  // namespace trit
