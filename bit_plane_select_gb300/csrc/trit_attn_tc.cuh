// Attention on the 5th-generation tensor cores: descriptors, products, tensor memory and
// waits shared by trit_attn_prefix.cu and trit_attn_prompt.cu.
#pragma once

#include <cuda.h>

#include "trit_attn.cuh"
#include "trit_tc.cuh"

namespace trit {
namespace attn {

using namespace tc;

constexpr int kBlockKeys = 128;    // keys of a tile of K or V

template <typename T>
__host__ __device__ constexpr uint32_t type_bits() { return 0; }
template <>
__host__ __device__ constexpr uint32_t type_bits<__nv_bfloat16>() { return (1u << 7) | (1u << 10); }

// Instruction descriptors, kind::f16, fp32 accumulator, M = 128: S (N = 128, both
// operands K-major) and O (N = D, B MN-major).
template <typename T>
__host__ __device__ constexpr uint32_t idesc_s() { return (1u << 4) | type_bits<T>() | ((128u >> 3) << 17) | ((128u >> 4) << 24); }
template <typename T, int D>
__host__ __device__ constexpr uint32_t idesc_o() {
    return (1u << 4) | type_bits<T>() | (1u << 16) | ((uint32_t(D) >> 3) << 17) | ((128u >> 4) << 24);
}

// Shared-memory matrix descriptors as two words: the start address and leading
// offset, and the stride (1024 bytes between groups of eight 128-byte rows),
// version and 128-byte swizzle.  A step along the operand adds to the first word
// only.  K-major (Q, K): the leading offset is unused.  MN-major (V as stored: 64
// columns of a key contiguous, 8 keys an atom): it is the distance of the
// next 64 columns, half a tile.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescK = 1u << 16, kDescMn = uint32_t((kBlockKeys * 128) >> 4) << 16;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return saddr >> 4; }

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(uint32_t(acc)), "r"(kDescHi));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n mov.b64 b, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(uint32_t(acc)), "r"(kDescHi));
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

// Waits for the phase of the given parity; false once *timed_out is set or kWaitNs
// have passed.  The clock is read every 256 tries only: a read of it
// takes longer than the waits here.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, uint32_t *timed_out) {
    unsigned long long t0 = 0;
    for (uint32_t i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 255) == 255) {
            if (*reinterpret_cast<volatile uint32_t *>(timed_out)) return false;
            const unsigned long long t = global_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitNs) {
                atomicExch(timed_out, 1u);
                return false;
            }
        }
    }
}

// Two fp32 lanes in one 64-bit register.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// Of a row with a far score (far_score): its scale becomes the power of two below it, and its base m_raw in that scale, so
// that weights are of exact differences from m_raw, the score that they are against.  (A score is known to a step there,
// which is four powers of two of a weight and more.)
__device__ __forceinline__ void far_scale(float m_raw, float &scale, float &base) {
    scale = __uint_as_float(__float_as_uint(scale) & 0x7f800000u);
    base = m_raw * scale;
}
// The same for a whole warp: one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint32_t *timed_out) {
    return __all_sync(~0u, bar_wait(bar, parity, timed_out));
}

#define TRIT_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define TRIT_W8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])

// 32 consecutive columns of the warp's 32 tensor-memory lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : TRIT_R8(v, 0), TRIT_R8(v, 8), TRIT_R8(v, 16), TRIT_R8(v, 24)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : TRIT_R8(v, 0), TRIT_R8(v, 8)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::
            TRIT_W8(v, 0),
        TRIT_W8(v, 8), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

}  // namespace attn
}  // namespace trit
