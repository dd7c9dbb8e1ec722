// trit_draft_verify: keep draft t while u_t q_t(x_t) < p_t(x_t); then
//     next = argmax_i r_i / e_i,   r = max(p_k - q_k, 0) or p,
// the winner of a race of exponential numbers e_i with rates r_i: P(i) =
// r_i / sum r without any sum over the vocabulary, so splitting the row over
// CTAs changes nothing in the answer.
//
// Bound by reading one row each of p, q and e (12 V bytes per sequence in
// fp32), or for few sequences by latency.  A cluster of eight CTAs takes a
// sequence: every CTA finds the first draft not kept by itself (two values per
// draft, one lane each) while its first race numbers are on their way, reads
// an eighth of the rows, and hands its best candidate -- a 64-bit key that
// orders by quotient and then by the lower index -- to the first CTA's shared
// memory, which writes the answer: no atomics, nothing kept between calls.
#include "trit_serve.cuh"

namespace trit {
namespace {

constexpr int kCluster = 8;
constexpr int kPer = 2;       // vectors of four of each row in flight per thread

// Threads of a CTA (NT): 256, six CTAs per SM, where there are sequences enough (192 of
// 131072 tokens: 48.7 us; 512 threads, four vectors, two CTAs: 58.5 -- a CTA reads
// nothing but race numbers until it knows its rows, so others have to); 512 and 1024
// where few CTAs have long rows (eight sequences of 131072: 7.9 us against 14.2; one of
// 32000, four vectors a thread already with 256: 4.9 against 4.1, so not there).

template <typename S>
__device__ __forceinline__ float as_f32(S v);
template <>
__device__ __forceinline__ float as_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float as_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Four values at element 4 i of a row: one load where the row is aligned for it.
template <typename S, bool VEC>
__device__ __forceinline__ float4 load4(const S *row, int64_t i) {
    if (!VEC) return make_float4(as_f32<S>(row[4 * i]), as_f32<S>(row[4 * i + 1]), as_f32<S>(row[4 * i + 2]),
                                 as_f32<S>(row[4 * i + 3]));
    if (sizeof(S) == 4) return __ldcs(reinterpret_cast<const float4 *>(row) + i);
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(row) + i);
    const S *s = reinterpret_cast<const S *>(&v);
    return make_float4(as_f32<S>(s[0]), as_f32<S>(s[1]), as_f32<S>(s[2]), as_f32<S>(s[3]));
}

// A lane's best candidate.  The quotient itself is formed only where the value can
// win: r/e > s needs r > s e, up to three roundings (1 - 2^-22 covers them) and
// the absolute error of a subnormal product (1e-37 covers it).  Candidates come in
// rising order of index, so the lowest of equal ones is kept.
struct Best {
    float s;
    uint32_t i;
    __device__ __forceinline__ void see(float r, float e, uint32_t at) {
        if (r > 0.0f && r + 1e-37f > (s * e) * (1.0f - 0x1p-22f)) {
            const float v = __fdiv_rn(r, e) + 0.0f;   // -0 becomes +0
            if (v > s && v >= 0.0f) {
                s = v;
                i = at;
            }
        }
    }
    __device__ __forceinline__ void see4(float4 r, float4 e, uint32_t at) {
        see(r.x, e.x, at);
        see(r.y, e.y, at + 1);
        see(r.z, e.z, at + 2);
        see(r.w, e.w, at + 3);
    }
};

// Candidates 4 i .. 4 i + 3 for i in [from, to), i = from + tid first; e0 holds the
// first kPer vectors of e.
template <typename S, bool VEC, int kThreads>
__device__ __forceinline__ void scan(Best &best, const S *p, const S *q, const float *e, int64_t from, int64_t to,
                                     int tid, float4 (&w)[kPer]) {
    for (int64_t i0 = from + tid; i0 < to; i0 += kThreads * kPer) {
        float4 a[kPer], b[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t i = i0 + k * kThreads < to ? i0 + k * kThreads : i0;   // again, not past the end
            a[k] = load4<S, VEC>(p, i);
            b[k] = q ? load4<S, VEC>(q, i) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t i = i0 + k * kThreads < to ? i0 + k * kThreads : i0;
            a[k].x -= b[k].x; a[k].y -= b[k].y; a[k].z -= b[k].z; a[k].w -= b[k].w;
            best.see4(a[k], w[k], uint32_t(4 * i));
        }
        const int64_t next = i0 + kThreads * kPer;
        if (next < to) {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                w[k] = load4<float, VEC>(e, next + k * kThreads < to ? next + k * kThreads : next);
        }
    }
}

__device__ __forceinline__ unsigned long long key_of(const Best &b) {
    return b.s < 0.0f ? 0ull
                      : (static_cast<unsigned long long>(__float_as_uint(b.s)) << 32) | (0xffffffffu - b.i);
}

template <int kThreads>
__device__ unsigned long long block_max(unsigned long long k, unsigned long long *sh) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const unsigned long long v = __shfl_xor_sync(~0u, k, o);
        k = v > k ? v : k;
    }
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = k;
    __syncthreads();
    k = sh[threadIdx.x & (kThreads / 32 - 1)];
#pragma unroll
    for (int o = kThreads / 64; o; o >>= 1) {
        const unsigned long long v = __shfl_xor_sync(~0u, k, o);
        k = v > k ? v : k;
    }
    __syncthreads();
    return k;
}

template <typename S, bool VEC, int kThreads>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, kThreads == 256 ? 6 : 1536 / kThreads)
    verify_kernel(const __grid_constant__ trit_verify_job J, uint32_t *err) {
    __shared__ unsigned long long sh[kThreads / 32];
    __shared__ unsigned long long keys[kCluster];     // in the first CTA: one per CTA
    __shared__ int sh_kept;
    const int b = blockIdx.x / kCluster, rank = blockIdx.x % kCluster, tid = threadIdx.x;
    // the first CTA's shared memory may be written once it is known to run: arrive here, wait before the store
    asm volatile("barrier.cluster.arrive.relaxed.aligned;");
    pdl_wait();
    pdl_launch();
    const S *P = static_cast<const S *>(J.p) + b * J.p_seq_stride;
    const S *Q = static_cast<const S *>(J.q) + b * J.q_seq_stride;
    const float *e = J.race + b * J.race_stride;
    const int64_t quads = J.V / 4, from = quads * rank / kCluster, to = quads * (rank + 1) / kCluster;
    float4 w[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int64_t i = from + tid + k * kThreads;
        w[k] = make_float4(1.f, 1.f, 1.f, 1.f);
        if (from + tid < to) w[k] = load4<float, VEC>(e, i < to ? i : from + tid);
    }
    int n = J.n_draft ? J.n_draft[b] : J.T;
    if (n < 0 || n > J.T) {
        if (tid == 0) raise_flag(err, TRIT_ERR_INDEX);
        n = n < 0 ? 0 : J.T;
    }
    if (tid < 32) {
        int kept = 0;
        for (int t0 = 0; t0 < n && kept == t0; t0 += 32) {
            const int t = t0 + tid;
            bool keep = false;
            if (t < n) {
                const int x = J.draft[int64_t(b) * J.T + t];
                const float u = J.u[int64_t(b) * J.T + t];
                if (x >= 0 && x < J.V) {
                    const float px = as_f32<S>(P[t * J.p_tok_stride + x]);
                    const float qx = as_f32<S>(Q[t * J.q_tok_stride + x]);
                    keep = __fmul_rn(u, qx) < px;
                } else {
                    raise_flag(err, TRIT_ERR_INDEX);
                }
            }
            const uint32_t lost = ~__ballot_sync(~0u, keep);
            kept += lost ? __ffs(int(lost)) - 1 : 32;
        }
        if (tid == 0) sh_kept = kept;
    }
    __syncthreads();
    const int kept = sh_kept;
    const S *p = P + kept * J.p_tok_stride;
    const S *q = kept < n ? Q + kept * J.q_tok_stride : nullptr;
    Best best{-1.0f, 0u};
    scan<S, VEC, kThreads>(best, p, q, e, from, to, tid, w);
    if (rank == kCluster - 1 && tid < J.V - 4 * quads) {      // the last V % 4
        const int64_t i = 4 * quads + tid;
        best.see(as_f32<S>(p[i]) - (q ? as_f32<S>(q[i]) : 0.0f), e[i], uint32_t(i));
    }
    unsigned long long key = block_max<kThreads>(key_of(best), sh);
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (tid == 0) {
        uint32_t to_first;
        asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to_first) : "r"(uint32_t(__cvta_generic_to_shared(&keys[rank]))));
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to_first), "l"(key) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;
    key = 0;
#pragma unroll
    for (int k = 0; k < kCluster; ++k) key = keys[k] > key ? keys[k] : key;
    if (key == 0 && q) {      // no candidate: where the residual is nowhere positive, p decides
        best = Best{-1.0f, 0u};
        int positive = 0;
        for (int64_t i = tid; i < J.V; i += kThreads) {
            const float pi = as_f32<S>(p[i]);
            positive |= pi - as_f32<S>(q[i]) > 0.0f;
            best.see(pi, e[i], uint32_t(i));
        }
        if (!__syncthreads_or(positive)) key = block_max<kThreads>(key_of(best), sh);
    }
    for (int t = tid; t <= J.T; t += kThreads) {
        int v = -1;
        if (t < kept) v = J.draft[int64_t(b) * J.T + t];
        if (t == kept && key) v = int(0xffffffffu - uint32_t(key));
        J.tokens[int64_t(b) * (J.T + 1) + t] = v;
    }
    if (tid == 0) {
        J.accepted[b] = kept;
        if (!key) raise_flag(err, TRIT_ERR_EMPTY);
    }
}

template <typename S, int NT>
cudaError_t launch_nt(const trit_verify_job &J, uint32_t *err, cudaStream_t s) {
    // vectors of four where every row starts on one
    auto on = [](const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
    const bool vec = on(J.p, 4 * sizeof(S)) && on(J.q, 4 * sizeof(S)) && on(J.race, 16) &&
                     ((J.p_seq_stride | J.p_tok_stride | J.q_seq_stride | J.q_tok_stride | J.race_stride) & 3) == 0;
    const dim3 grid(unsigned(J.B) * kCluster), block(NT);
    return vec ? launch_pdl(verify_kernel<S, true, NT>, grid, block, 0, s, J, err)
               : launch_pdl(verify_kernel<S, false, NT>, grid, block, 0, s, J, err);
}
template <typename S>
cudaError_t launch(const trit_verify_job &J, uint32_t *err, cudaStream_t s) {
    const int64_t sms = device_sm_count(), ctas = int64_t(J.B) * kCluster;
    if (J.V <= 65536 || ctas > 2 * sms) return launch_nt<S, 256>(J, err, s);
    return ctas <= sms ? launch_nt<S, 1024>(J, err, s) : launch_nt<S, 512>(J, err, s);
}

}  // namespace

cudaError_t launch_draft_verify(const trit_verify_job &J, uint32_t *err, cudaStream_t s) {
    return J.dtype == TRIT_F32    ? launch<float>(J, err, s)
           : J.dtype == TRIT_BF16 ? launch<__nv_bfloat16>(J, err, s)
                                  : launch<__half>(J, err, s);
}

}  // namespace trit
