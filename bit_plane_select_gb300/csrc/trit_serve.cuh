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

// W consecutive values of a row, and their store.
template <int W>
__device__ __forceinline__ void load_row(const float *p, float (&x)[W]) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p + i));
        x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
}
template <int W, typename H>
__device__ __forceinline__ void load_row(const H *p, float (&x)[W]) {
    uint32_t w[W / 2];
    if (W == 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = v.x; w[1] = v.y; w[W / 2 - 2] = v.z; w[W / 2 - 1] = v.w;
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x; w[1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        const float2 f = unpack16<H>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <int W, typename T>
__device__ __forceinline__ void store_row(T *p, const float (&y)[W]) {
    uint32_t w[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) w[i] = pack16<T>(y[2 * i], y[2 * i + 1]);
    if (W == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[W / 2 - 2], w[W / 2 - 1]);
    else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// The sequence that packed row `row` may belong to: the last b < B with starts[b] <= row, or -1.
// 32 starts at a time; a whole warp asks for one row.  (Starts that fall give some b
// in range: the caller checks the row against that sequence's own starts.)
__device__ __forceinline__ int sequence_of(const int32_t *starts, int B, int64_t row, int lane) {
    int lo = 0, n = B;
    for (;;) {
        const int step = (n + 31) / 32, at = lane * step;
        const uint32_t before = __ballot_sync(~0u, at < n && starts[lo + (at < n ? at : 0)] <= row);
        if (!before) return -1;
        const int k = 31 - __clz(int(before));
        lo += k * step;
        n = n - k * step < step ? n - k * step : step;
        if (step == 1) return lo;
    }
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
