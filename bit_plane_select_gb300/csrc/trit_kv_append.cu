// trit_kv_append: per head vector x of a new token's q and k (fp32 arithmetic)
//     y = x / sqrt(mean(x^2) + eps) * g          (where there is a gain g)
//     (a, b) <- (a c - b s, b c + a s)            c, s = cos, sin[position][j]
// over the first `rot` columns, rounded once to the cache's type: q into q_out,
// k into the token's cache slot, v copied into it.
//
// A stream of (Hq + 2 Hkv) D values per token, each read once and written
// once: bound by memory for many tokens and by the latency of three dependent
// loads (lengths, page id and table rows) for few.  A lane holds eight (four)
// consecutive columns of a vector, so a warp takes two vectors of D = 128 per
// step, four of 64; a rotation partner is then a fixed number of lanes away
// (rot/2 columns) and the norm is a shuffle sum.  Instructions count as well: at
// 32768 tokens of 30 vectors with norms, four columns a lane took 168 us and eight
// take 121 (6.4 TB/s).
#include "trit_serve.cuh"

namespace trit {
namespace {

constexpr int kThreads = 128;
// Warp steps of a warp, all in flight together (measured at 32768 tokens of 30 vectors,
// eight columns a lane: 2 steps 148 us, 3 steps 130, 5 steps 121).
constexpr int kGroups = 5;

struct AppendArgs {
    trit_kv_append_job J;
    uint32_t *err;
    int32_t chunks;      // warps per token
    int32_t page_shift;  // log2(page_size), or -1
};

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

template <typename T, typename S, int D, bool PAIRS, int W>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs A) {
    const trit_kv_append_job &J = A.J;
    static_assert(W == 8 || (W == 4 && !PAIRS), "angles are read four at a time");
    constexpr int L = D / W;             // lanes of one head vector
    constexpr int V = 32 / L;            // vectors of a warp step
    const int lane = threadIdx.x & 31, sub = lane % L, which = lane / L;
    const int warp = int(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);    // < 2^31
    const int token = warp / A.chunks;
    pdl_wait();
    pdl_launch();
    if (token >= J.batch.B * J.batch.T) return;
    const int first = (warp - token * A.chunks) * kGroups;
    const int b = token / J.batch.T, t = token - b * J.batch.T;
    const int Hq = J.q ? J.q_heads : 0, Hkv = J.cache.heads, all = Hq + 2 * Hkv;
    const int j0 = sub * W, half = J.rot / 2;

    // every value first: the rest of the token's loads depend on one another
    const S *qp = static_cast<const S *>(J.q) + token * J.q_stride + j0;
    const S *kp = static_cast<const S *>(J.k) + token * J.k_stride + j0 - Hq * D;
    const S *vp = static_cast<const S *>(J.v) + token * J.v_stride + j0 - (Hq + Hkv) * D;
    float x[kGroups][W];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        int h = (first + g) * V + which;                    // vector of the token: q, k, v heads in turn
        h = h < all ? h : all - 1;
        load_row<W>((h < Hq ? qp : h < Hq + Hkv ? kp : vp) + h * D, x[g]);
    }

    // where the token goes
    const int len = J.batch.lens[b], given = J.batch.new_lens ? J.batch.new_lens[b] : J.batch.T;
    const int n = given < 0 ? 0 : given < J.batch.T ? given : J.batch.T;
    const int64_t own = int64_t(len) - n + t;
    const int64_t pos = J.batch.prefix_len + own;
    bool ok = t < n;
    int64_t slot_at = 0;
    const bool turns = j0 < J.rot;
    constexpr int CW = PAIRS ? W / 2 : W;
    float c[CW], s[CW];
#pragma unroll
    for (int i = 0; i < CW; ++i) {
        c[i] = 1.0f;
        s[i] = 0.0f;
    }
    if (ok) {
        const bool in = own >= 0 && (J.rot == 0 || pos < J.max_pos);
        // the lane's angles, and the page beside them
        if (in && turns) {
            const int64_t at = pos * half + (PAIRS ? j0 / 2 : j0 < half ? j0 : j0 - half);
            load_row<CW>(J.cos + at, c);
            load_row<CW>(J.sin + at, s);
        }
        const int64_t col = own < 0 ? -1 : A.page_shift >= 0 ? own >> A.page_shift : own / J.cache.page_size;
        int page = -1;
        if (in && col < J.batch.table_pages) page = J.batch.table[b * J.batch.table_stride + col];
        ok = page >= 0 && page < J.cache.pages;
        if (!ok) raise_flag(A.err, TRIT_ERR_INDEX);
        slot_at = page * J.cache.page_stride + (own - col * J.cache.page_size) * J.cache.slot_stride;
    }
    // the lane holding the rotation partners, and the sign of their sine (rot / 2 is a
    // multiple of W here)
    const int partner = !turns ? lane : (j0 < half ? lane + half / W : lane - half / W);
    if (!PAIRS && j0 < half) {
#pragma unroll
        for (int i = 0; i < CW; ++i) s[i] = -s[i];
    }
    T *q_out = static_cast<T *>(J.q_out) + int64_t(token) * Hq * D + j0;
    T *k_out = static_cast<T *>(J.cache.k) + slot_at + j0;
    T *v_out = static_cast<T *>(J.cache.v) + slot_at + j0;

#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int h = (first + g) * V + which;
        const bool is_q = h < Hq, is_v = h >= Hq + Hkv;
        float(&v)[W] = x[g];
        if (J.q_gain || J.k_gain) {                         // uniform: every lane shuffles
            float sum = v[0] * v[0];
#pragma unroll
            for (int i = 1; i < W; ++i) sum = fmaf(v[i], v[i], sum);
#pragma unroll
            for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            const float *gain = is_q ? J.q_gain : is_v ? nullptr : J.k_gain;
            if (gain) {
                const float r = rsqrtf(sum * (1.0f / D) + J.eps);
                float gg[W];
                load_row<W>(gain + j0, gg);
#pragma unroll
                for (int i = 0; i < W; ++i) v[i] = v[i] * r * gg[i];
            }
        }
        if (PAIRS) {
            if (turns && !is_v) {
#pragma unroll
                for (int i = 0; i < W / 2; ++i) {
                    const float a0 = v[2 * i], a1 = v[2 * i + 1];
                    v[2 * i] = a0 * c[i % CW] - a1 * s[i % CW];
                    v[2 * i + 1] = a1 * c[i % CW] + a0 * s[i % CW];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float o = __shfl_sync(~0u, v[i], partner);
                if (turns && !is_v) v[i] = v[i] * c[i % CW] + o * s[i % CW];
            }
        }
        if (h >= all || (!ok && !is_q)) continue;
        if (!ok) {                                          // a padding token's query
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = 0.0f;
        }
        store_row<W>(is_q ? q_out + h * D
                          : is_v ? v_out + (h - Hq - Hkv) * J.cache.head_stride
                                 : k_out + (h - Hq) * J.cache.head_stride,
                     v);
    }
    // (up there a branch on it would part the loads: 32768 tokens 159 us instead of 121)
    if (n != given) raise_flag(A.err, TRIT_ERR_INDEX);
}

template <typename T, typename S, int D>
cudaError_t launch_d(const AppendArgs &A, int W, int64_t blocks, cudaStream_t s) {
    const dim3 grid{unsigned(blocks)}, block{kThreads};
    if (A.J.flags & TRIT_ROPE_PAIRS) return launch_pdl(append_kernel<T, S, D, true, 8>, grid, block, 0, s, A);
    return W == 8 ? launch_pdl(append_kernel<T, S, D, false, 8>, grid, block, 0, s, A)
                  : launch_pdl(append_kernel<T, S, D, false, 4>, grid, block, 0, s, A);
}
template <typename T, typename S>
cudaError_t launch_s(const AppendArgs &A, int W, int64_t blocks, cudaStream_t s) {
    return A.J.cache.head_dim == 128 ? launch_d<T, S, 128>(A, W, blocks, s) : launch_d<T, S, 64>(A, W, blocks, s);
}

}  // namespace

cudaError_t launch_kv_append(const trit_kv_append_job &J, uint32_t *err, cudaStream_t s) {
    AppendArgs A;
    A.J = J;
    A.err = err;
    const int vectors = (J.q ? J.q_heads : 0) + 2 * J.cache.heads;
    // eight columns a lane, except where halves of the rotation do not start on eight
    const int W = (J.flags & TRIT_ROPE_PAIRS) || J.rot % 16 == 0 ? 8 : 4;
    const int per_step = 32 * W / J.cache.head_dim;
    const int steps = (vectors + per_step - 1) / per_step;
    A.chunks = (steps + kGroups - 1) / kGroups;
    A.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (J.cache.page_size == (1 << i)) A.page_shift = i;
    const int64_t warps = int64_t(J.batch.B) * J.batch.T * A.chunks;
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (J.cache.dtype == TRIT_BF16)
        return J.src_dtype == TRIT_F32 ? launch_s<__nv_bfloat16, float>(A, W, blocks, s)
                                       : launch_s<__nv_bfloat16, __nv_bfloat16>(A, W, blocks, s);
    return J.src_dtype == TRIT_F32 ? launch_s<__half, float>(A, W, blocks, s)
                                   : launch_s<__half, __half>(A, W, blocks, s);
}

}  // namespace trit
