// trit_draft_verify: keep draft t while u_t q_t(x_t) < p_t(x_t); then
//     next = argmax_i r_i / e_i,   r = max(p_k - q_k, 0) or p,
// the winner of a race of exponential numbers e_i with rates r_i: P(i) =
// r_i / sum r without any sum over the vocabulary, so splitting the row over
// CTAs changes nothing in the answer.
//
// Bound by reading one row each of p, q and e (12 V bytes per sequence in
// fp32).  A row is cut into chunks, one CTA each; every CTA finds the first
// draft not kept by itself (two values per draft, one lane each), and the
// CTAs of a sequence meet in one 64-bit maximum whose key orders by quotient
// and then by the lower index.  The last CTA to arrive writes the answer and
// leaves the workspace zeroed.
#include "trit_serve.cuh"

namespace trit {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;      // values of each row in flight per thread

struct Slot {                  // workspace of one sequence
    unsigned long long best;   // (quotient bits << 32) | ~index; 0: no candidate yet
    uint32_t arrived;
    uint32_t pad_;
};

template <typename S>
__device__ __forceinline__ float as_f32(S v);
template <>
__device__ __forceinline__ float as_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float as_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// A lane's best candidate.  The quotient itself is formed only where the value can
// win: r/e > s needs r > s e, up to three roundings (1 - 2^-22 covers them) and
// the absolute error of a subnormal product (1e-37 covers it).
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
};

template <typename S>
__device__ Best scan(const S *p, const S *q, const float *e, int64_t from, int64_t to, int tid) {
    Best best{-1.0f, 0u};
    for (int64_t i0 = from; i0 < to; i0 += kThreads * kPer) {
        float r[kPer], w[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t i = i0 + k * kThreads + tid;
            r[k] = 0.0f;
            w[k] = 1.0f;
            if (i < to) {
                r[k] = as_f32<S>(p[i]);
                if (q) r[k] -= as_f32<S>(q[i]);
                w[k] = e[i];
            }
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) best.see(r[k], w[k], uint32_t(i0 + k * kThreads + tid));
    }
    return best;
}

__device__ __forceinline__ unsigned long long key_of(const Best &b) {
    return b.s < 0.0f ? 0ull
                      : (static_cast<unsigned long long>(__float_as_uint(b.s)) << 32) | (0xffffffffu - b.i);
}

__device__ unsigned long long block_max(unsigned long long k, unsigned long long *sh) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const unsigned long long v = __shfl_xor_sync(~0u, k, o);
        k = v > k ? v : k;
    }
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = k;
    __syncthreads();
    k = sh[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) k = sh[w] > k ? sh[w] : k;
    __syncthreads();
    return k;
}

template <typename S>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ trit_verify_job J,
                                                          uint32_t *err, int64_t chunk) {
    __shared__ unsigned long long sh[kThreads / 32];
    __shared__ int sh_kept;
    __shared__ bool sh_last;
    const int b = blockIdx.y, tid = threadIdx.x;
    const S *P = static_cast<const S *>(J.p) + b * J.p_seq_stride;
    const S *Q = static_cast<const S *>(J.q) + b * J.q_seq_stride;
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
                if (x >= 0 && x < J.V) {
                    const float px = as_f32<S>(P[t * J.p_tok_stride + x]);
                    const float qx = as_f32<S>(Q[t * J.q_tok_stride + x]);
                    keep = __fmul_rn(J.u[int64_t(b) * J.T + t], qx) < px;
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
    const float *e = J.race + b * J.race_stride;
    const int64_t from = blockIdx.x * chunk, to = from + chunk < J.V ? from + chunk : J.V;
    unsigned long long key = block_max(key_of(scan<S>(p, q, e, from, to, tid)), sh);
    Slot *slot = static_cast<Slot *>(J.workspace) + b;
    if (tid == 0) {
        if (key) atomicMax(&slot->best, key);
        __threadfence();
        sh_last = atomicAdd(&slot->arrived, 1u) + 1 == gridDim.x;
    }
    __syncthreads();
    if (!sh_last) return;
    __threadfence();
    key = *reinterpret_cast<volatile unsigned long long *>(&slot->best);
    if (key == 0 && q) key = block_max(key_of(scan<S>(p, nullptr, e, 0, J.V, tid)), sh);
    for (int t = tid; t <= J.T; t += kThreads) {
        int v = -1;
        if (t < kept) v = J.draft[int64_t(b) * J.T + t];
        if (t == kept && key) v = int(0xffffffffu - uint32_t(key));
        J.tokens[int64_t(b) * (J.T + 1) + t] = v;
    }
    if (tid == 0) {
        J.accepted[b] = kept;
        if (!key) raise_flag(err, TRIT_ERR_EMPTY);
        slot->best = 0;
        slot->arrived = 0;
    }
}

}  // namespace

cudaError_t launch_draft_verify(const trit_verify_job &J, uint32_t *err, cudaStream_t s) {
    const int64_t step = kThreads * kPer;
    const int64_t most = (J.V + step - 1) / step;                    // chunks of one load round
    int64_t chunks = (int64_t(device_sm_count()) * 8 + J.B - 1) / J.B;
    if (chunks > most) chunks = most;
    const int64_t rounds = (most + chunks - 1) / chunks;
    const int64_t chunk = rounds * step;
    const dim3 grid(unsigned((J.V + chunk - 1) / chunk), unsigned(J.B));
    if (J.dtype == TRIT_F32)
        verify_kernel<float><<<grid, kThreads, 0, s>>>(J, err, chunk);
    else if (J.dtype == TRIT_BF16)
        verify_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(J, err, chunk);
    else
        verify_kernel<__half><<<grid, kThreads, 0, s>>>(J, err, chunk);
    return cudaGetLastError();
}

}  // namespace trit
