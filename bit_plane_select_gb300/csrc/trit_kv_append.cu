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

struct AppendArgs {
    trit_kv_append_job J;
    uint32_t *err;
    int32_t steps;       // vector groups per token
    int32_t per_warp;    // groups one warp takes
    int32_t chunks;      // warps per token
    int32_t pad_;
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
    const int64_t warp = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t token = warp / A.chunks;
    if (token >= int64_t(J.batch.B) * J.batch.T) return;
    const int first = int(warp - token * A.chunks) * A.per_warp;
    const int b = int(token / J.batch.T), t = int(token - int64_t(b) * J.batch.T);
    const int Hq = J.q ? J.q_heads : 0, Hkv = J.cache.heads;

    // where the token goes
    const int n = batch_new(J.batch, b);
    const int64_t own = int64_t(J.batch.lens[b]) - n + t;
    const int64_t pos = J.batch.prefix_len + own;
    bool ok = t < n;
    int64_t slot_at = 0;
    if (ok) {
        const int64_t col = own >= 0 ? own / J.cache.page_size : -1;
        int page = -1;
        if (col >= 0 && col < J.batch.table_pages) page = J.batch.table[b * J.batch.table_stride + col];
        ok = page >= 0 && page < J.cache.pages && (J.rot == 0 || pos < J.max_pos);
        if (!ok) raise_flag(A.err, TRIT_ERR_INDEX);
        slot_at = page * J.cache.page_stride + (own - col * J.cache.page_size) * J.cache.slot_stride;
    }
    // the lane's angles
    const int j0 = sub * 4, half = J.rot / 2;
    const bool turns = j0 < J.rot;
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (ok && turns) {
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
    // the lane holding the rotation partners, and the sign of their sine
    const int partner = !turns ? lane : (j0 < half ? lane + half / 4 : lane - half / 4);
    const float sign = j0 < half ? -1.f : 1.f;

    const int last = first + A.per_warp < A.steps ? first + A.per_warp : A.steps;
    for (int g = first; g < last; ++g) {
        const int h = g * V + which;                        // vector of the token: q, k, v heads in turn
        const bool is_q = h < Hq, is_k = !is_q && h < Hq + Hkv, live = h < Hq + 2 * Hkv;
        const int hk = h - Hq - (is_k ? 0 : Hkv);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live && ok) {
            const S *p = is_q ? static_cast<const S *>(J.q) + token * J.q_stride + int64_t(h) * D
                       : is_k ? static_cast<const S *>(J.k) + token * J.k_stride + int64_t(hk) * D
                              : static_cast<const S *>(J.v) + token * J.v_stride + int64_t(hk) * D;
            x = Src<S>::load4(p + j0);
        }
        const float *gain = is_q ? J.q_gain : is_k ? J.k_gain : nullptr;
        float sum = x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w;
        if (J.q_gain || J.k_gain) {                         // uniform: every lane shuffles
#pragma unroll
            for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        }
        if (gain) {
            const float r = __frsqrt_rn(sum * (1.0f / D) + J.eps);
            const float4 gg = __ldg(reinterpret_cast<const float4 *>(gain + j0));
            x.x = x.x * r * gg.x; x.y = x.y * r * gg.y; x.z = x.z * r * gg.z; x.w = x.w * r * gg.w;
        }
        float4 y = x;
        if (PAIRS) {
            if (turns && (is_q || is_k)) {
                y.x = x.x * c[0] - x.y * s[0];
                y.y = x.y * c[1] + x.x * s[1];
                y.z = x.z * c[2] - x.w * s[2];
                y.w = x.w * c[3] + x.z * s[3];
            }
        } else {
            float4 o;
            o.x = __shfl_sync(~0u, x.x, partner);
            o.y = __shfl_sync(~0u, x.y, partner);
            o.z = __shfl_sync(~0u, x.z, partner);
            o.w = __shfl_sync(~0u, x.w, partner);
            if (turns && (is_q || is_k)) {
                y.x = x.x * c[0] + sign * (o.x * s[0]);
                y.y = x.y * c[1] + sign * (o.y * s[1]);
                y.z = x.z * c[2] + sign * (o.z * s[2]);
                y.w = x.w * c[3] + sign * (o.w * s[3]);
            }
        }
        if (!live || (!ok && !is_q)) continue;
        T *out = is_q ? static_cast<T *>(J.q_out) + (token * Hq + h) * D
                      : static_cast<T *>(is_k ? J.cache.k : J.cache.v) + slot_at + hk * J.cache.head_stride;
        *reinterpret_cast<uint2 *>(out + j0) = make_uint2(pack16<T>(y.x, y.y), pack16<T>(y.z, y.w));
    }
}

template <typename T, typename S, int D>
cudaError_t launch_d(const AppendArgs &A, int64_t blocks, cudaStream_t s) {
    if (A.J.flags & TRIT_ROPE_PAIRS)
        append_kernel<T, S, D, true><<<dim3(unsigned(blocks)), kThreads, 0, s>>>(A);
    else
        append_kernel<T, S, D, false><<<dim3(unsigned(blocks)), kThreads, 0, s>>>(A);
    return cudaGetLastError();
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
    A.steps = (vectors + per_step - 1) / per_step;
    A.per_warp = 5;
    A.chunks = (A.steps + A.per_warp - 1) / A.per_warp;
    A.pad_ = 0;
    const int64_t warps = int64_t(J.batch.B) * J.batch.T * A.chunks;
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (J.cache.dtype == TRIT_BF16)
        return J.src_dtype == TRIT_F32 ? launch_s<__nv_bfloat16, float>(A, blocks, s)
                                       : launch_s<__nv_bfloat16, __nv_bfloat16>(A, blocks, s);
    return J.src_dtype == TRIT_F32 ? launch_s<__half, float>(A, blocks, s)
                                   : launch_s<__half, __half>(A, blocks, s);
}

}  // namespace trit
