// trit_kv_append: per head vector x of a new token's q and k (fp32 arithmetic)
//     y = x / sqrt(mean(x^2) + eps) * g          (where there is a gain g)
//     (a, b) <- (a c - b s, b c + a s)            c, s = cos, sin[position][j]
// over the first `rot` columns, rounded once to the cache's type: q into q_out,
// k into the token's cache slot, v copied into it.
//
// A stream of (Hq + 2 Hkv) D values per token, each read once and written
// once: bound by memory for many tokens and by the latency of three dependent
// loads (lengths, page id and table rows) for few.  A lane holds four
// consecutive columns of a vector, so a warp takes 128 columns (one vector of
// D = 128, two of 64) per step; a rotation partner is then a fixed number of
// lanes away (rot/2 columns = rot/8 lanes) and the norm is a shuffle sum.
#include "trit_serve.cuh"

namespace trit {
namespace {

constexpr int kThreads = 128;
constexpr int kGroups = 5;    // vector groups of a warp, all in flight together

struct AppendArgs {
    trit_kv_append_job J;
    uint32_t *err;
    int32_t chunks;      // warps per token
    int32_t page_shift;  // log2(page_size), or -1
};

template <typename S>
struct Src;
template <>
struct Src<float> {
    static __device__ __forceinline__ float4 load4(const float *p) {
        return __ldg(reinterpret_cast<const float4 *>(p));
    }
};
template <typename H>
struct Src16 {
    static __device__ __forceinline__ float4 load4(const H *p) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        const float2 a = unpack16<H>(v.x), b = unpack16<H>(v.y);
        return make_float4(a.x, a.y, b.x, b.y);
    }
};
template <>
struct Src<__half> : Src16<__half> {};
template <>
struct Src<__nv_bfloat16> : Src16<__nv_bfloat16> {};

template <typename T, typename S, int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs A) {
    const trit_kv_append_job &J = A.J;
    constexpr int L = D / 4;             // lanes of one head vector
    constexpr int V = 32 / L;            // vectors of a warp step
    const int lane = threadIdx.x & 31, sub = lane % L, which = lane / L;
    const int warp = int(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);    // < 2^24 tokens * chunks
    const int token = warp / A.chunks;
    pdl_wait();
    pdl_launch();
    if (token >= J.batch.B * J.batch.T) return;
    const int first = (warp - token * A.chunks) * kGroups;
    const int b = token / J.batch.T, t = token - b * J.batch.T;
    const int Hq = J.q ? J.q_heads : 0, Hkv = J.cache.heads, all = Hq + 2 * Hkv;
    const int j0 = sub * 4, half = J.rot / 2;

    // every value first: the rest of the token's loads depend on one another
    float4 x[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        int h = (first + g) * V + which;                    // vector of the token: q, k, v heads in turn
        h = h < all ? h : all - 1;
        const bool is_q = h < Hq, is_k = h < Hq + Hkv;
        const int hk = h - Hq - (is_k ? 0 : Hkv);
        const S *p = is_q ? static_cast<const S *>(J.q) + token * J.q_stride + h * D
                   : is_k ? static_cast<const S *>(J.k) + token * J.k_stride + hk * D
                          : static_cast<const S *>(J.v) + token * J.v_stride + hk * D;
        x[g] = Src<S>::load4(p + j0);
    }

    // where the token goes
    const int len = J.batch.lens[b], n = batch_new(J.batch, b);
    const int64_t own = int64_t(len) - n + t;
    const int64_t pos = J.batch.prefix_len + own;
    bool ok = t < n;
    int64_t slot_at = 0;
    const bool turns = j0 < J.rot;
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (ok) {
        const bool in = own >= 0 && (J.rot == 0 || pos < J.max_pos);
        // the lane's angles, and the page beside them
        if (in && turns) {
            if (PAIRS) {
                const float2 cc = __ldg(reinterpret_cast<const float2 *>(J.cos + pos * half + j0 / 2));
                const float2 ss = __ldg(reinterpret_cast<const float2 *>(J.sin + pos * half + j0 / 2));
                c[0] = c[1] = cc.x; c[2] = c[3] = cc.y;
                s[0] = s[1] = ss.x; s[2] = s[3] = ss.y;
            } else {
                const int j = j0 < half ? j0 : j0 - half;
                const float4 cc = __ldg(reinterpret_cast<const float4 *>(J.cos + pos * half + j));
                const float4 ss = __ldg(reinterpret_cast<const float4 *>(J.sin + pos * half + j));
                c[0] = cc.x; c[1] = cc.y; c[2] = cc.z; c[3] = cc.w;
                s[0] = ss.x; s[1] = ss.y; s[2] = ss.z; s[3] = ss.w;
            }
        }
        const int64_t col = own < 0 ? -1 : A.page_shift >= 0 ? own >> A.page_shift : own / J.cache.page_size;
        int page = -1;
        if (in && col < J.batch.table_pages) page = J.batch.table[b * J.batch.table_stride + col];
        ok = page >= 0 && page < J.cache.pages;
        if (!ok) raise_flag(A.err, TRIT_ERR_INDEX);
        slot_at = page * J.cache.page_stride + (own - col * J.cache.page_size) * J.cache.slot_stride;
    }
    // the lane holding the rotation partners, and the sign of their sine
    const int partner = !turns ? lane : (j0 < half ? lane + half / 4 : lane - half / 4);
    const float sign = j0 < half ? -1.f : 1.f;

#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int h = (first + g) * V + which;
        const bool is_q = h < Hq, is_k = !is_q && h < Hq + Hkv, live = h < all;
        const int hk = h - Hq - (is_k ? 0 : Hkv);
        float4 v = x[g];
        const float *gain = is_q ? J.q_gain : is_k ? J.k_gain : nullptr;
        if (J.q_gain || J.k_gain) {                         // uniform: every lane shuffles
            float sum = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
            for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            if (gain) {
                const float r = __frsqrt_rn(sum * (1.0f / D) + J.eps);
                const float4 gg = __ldg(reinterpret_cast<const float4 *>(gain + j0));
                v.x = v.x * r * gg.x; v.y = v.y * r * gg.y; v.z = v.z * r * gg.z; v.w = v.w * r * gg.w;
            }
        }
        float4 y = v;
        if (PAIRS) {
            if (turns && (is_q || is_k)) {
                y.x = v.x * c[0] - v.y * s[0];
                y.y = v.y * c[1] + v.x * s[1];
                y.z = v.z * c[2] - v.w * s[2];
                y.w = v.w * c[3] + v.z * s[3];
            }
        } else {
            float4 o;
            o.x = __shfl_sync(~0u, v.x, partner);
            o.y = __shfl_sync(~0u, v.y, partner);
            o.z = __shfl_sync(~0u, v.z, partner);
            o.w = __shfl_sync(~0u, v.w, partner);
            if (turns && (is_q || is_k)) {
                y.x = v.x * c[0] + sign * (o.x * s[0]);
                y.y = v.y * c[1] + sign * (o.y * s[1]);
                y.z = v.z * c[2] + sign * (o.z * s[2]);
                y.w = v.w * c[3] + sign * (o.w * s[3]);
            }
        }
        if (!live || (!ok && !is_q)) continue;
        if (!ok) y = make_float4(0.f, 0.f, 0.f, 0.f);       // a padding token's query
        T *out = is_q ? static_cast<T *>(J.q_out) + (int64_t(token) * Hq + h) * D
                      : static_cast<T *>(is_k ? J.cache.k : J.cache.v) + slot_at + hk * J.cache.head_stride;
        *reinterpret_cast<uint2 *>(out + j0) = make_uint2(pack16<T>(y.x, y.y), pack16<T>(y.z, y.w));
    }
}

template <typename T, typename S, int D>
cudaError_t launch_d(const AppendArgs &A, int64_t blocks, cudaStream_t s) {
    if (A.J.flags & TRIT_ROPE_PAIRS)
        return launch_pdl(append_kernel<T, S, D, true>, dim3(unsigned(blocks)), dim3(kThreads), 0, s, A);
    return launch_pdl(append_kernel<T, S, D, false>, dim3(unsigned(blocks)), dim3(kThreads), 0, s, A);
}
template <typename T, typename S>
cudaError_t launch_s(const AppendArgs &A, int64_t blocks, cudaStream_t s) {
    return A.J.cache.head_dim == 128 ? launch_d<T, S, 128>(A, blocks, s) : launch_d<T, S, 64>(A, blocks, s);
}

}  // namespace

cudaError_t launch_kv_append(const trit_kv_append_job &J, uint32_t *err, cudaStream_t s) {
    AppendArgs A;
    A.J = J;
    A.err = err;
    const int vectors = (J.q ? J.q_heads : 0) + 2 * J.cache.heads;
    const int per_step = J.cache.head_dim == 128 ? 1 : 2;
    const int steps = (vectors + per_step - 1) / per_step;
    A.chunks = (steps + kGroups - 1) / kGroups;
    A.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (J.cache.page_size == (1 << i)) A.page_shift = i;
    const int64_t warps = int64_t(J.batch.B) * J.batch.T * A.chunks;
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (J.cache.dtype == TRIT_BF16)
        return J.src_dtype == TRIT_F32 ? launch_s<__nv_bfloat16, float>(A, blocks, s)
                                       : launch_s<__nv_bfloat16, __nv_bfloat16>(A, blocks, s);
    return J.src_dtype == TRIT_F32 ? launch_s<__half, float>(A, blocks, s)
                                   : launch_s<__half, __half>(A, blocks, s);
}

}  // namespace trit
