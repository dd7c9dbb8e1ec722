// trit_logprobs: of a row x of V logits, with m = max x and l = sum e^(x - m),
//     logprob = x[token] - m - ln l,  entropy = ln l - (sum e^(x - m) (x - m)) / l,
// and the top_n largest x, lower indices first among equals.
//
// One pass: a thread keeps (m, l, w = sum e^(x - m) (x - m)) of what it has seen; when
// its maximum moves from m to m' they become f l and f (w + (m - m') l), f = e^(m - m').
// Both terms of the entropy are positive, so nothing cancels.
//
// The top entries need no second pass over the row.  Order entries by (value, lower
// index) and, coarser, by (value, lower chunk of 16 bytes).  A thread knows its greatest
// entry in the coarse order from the running maximum for nothing; the top_n-th of the
// 64 groups' greatest (a few threads each) is a bound that at least top_n
// entries reach, so an entry below it is none of the answer.  Only the threads that reach it --
// little more than top_n of 256 -- have their chunks read again, and the few dozen entries
// found are ranked by counting.  (Where more than kRoom are found, which takes values
// that lie by stride, top_n passes find one entry each.)
//
// Bound by reading the logits once, or for few rows by latency: then a cluster of up to
// eight CTAs shares a row, and the first of them joins (m, l, w) and ranks the CTAs'
// own top entries, handed over in its shared memory.
#include "trit_serve.cuh"

namespace trit {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 4;                   // an SM
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = 64;                // at least TRIT_MAX_TOP
constexpr int kMaxCluster = 8;
constexpr int kRoom = 2048;                // entries that may reach the bound
constexpr int kFlight = 4;                 // chunks of a thread in flight
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kGroups >= TRIT_MAX_TOP, "a bound needs a group for each entry");

typedef unsigned long long u64;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The greater, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Two fp32 lanes in one 64-bit register: one instruction for both.
__device__ __forceinline__ u64 pack2(float x, float y) {
    u64 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 unpack2(u64 v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
    u64 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
    u64 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
    u64 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// The greatest of 16 bytes of logits (NaN if one is), 16-bit ones two at a time.
template <typename S>
__device__ __forceinline__ float greatest(uint4 u);
template <>
__device__ __forceinline__ float greatest<float>(uint4 u) {
    float d;
    asm("{\n .reg .f32 t;\n max.NaN.f32 t, %1, %2, %3;\n max.NaN.f32 %0, t, %4;\n}"
        : "=f"(d)
        : "f"(__uint_as_float(u.x)), "f"(__uint_as_float(u.y)), "f"(__uint_as_float(u.z)), "f"(__uint_as_float(u.w)));
    return d;
}
#define TRIT_GREATEST(S, type)                                                                                       \
    template <>                                                                                                      \
    __device__ __forceinline__ float greatest<S>(uint4 u) {                                                          \
        uint32_t d;                                                                                                  \
        asm("{\n .reg .b32 s, t;\n max.NaN." type " s, %1, %2;\n max.NaN." type " t, %3, %4;\n max.NaN." type " %0, s, t;\n}" \
            : "=r"(d)                                                                                                \
            : "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w));                                                               \
        const float2 f = unpack16<S>(d);                                                                             \
        return max_nan(f.x, f.y);                                                                                    \
    }
TRIT_GREATEST(__nv_bfloat16, "bf16x2")
TRIT_GREATEST(__half, "f16x2")
#undef TRIT_GREATEST

// A float as a whole number of the same order (-0 as +0); -inf and NaN are not asked for.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ u64 key_of(float x, uint32_t at) {
    return x == -INFINITY ? 0ull : (u64(order_of(x)) << 32) | (0xffffffffu - at);
}

template <typename S>
__device__ __forceinline__ float to_f32(S v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// A row as chunks of 16 aligned bytes: chunk c holds the entries c E - off .. + E - 1, those
// outside the row read as -inf.
template <typename S>
struct Row {
    static constexpr int E = 16 / sizeof(S);
    const S *x;
    int64_t V;
    int off;           // entries of chunk 0 before the row
    uint32_t chunks;
    __device__ __forceinline__ Row(const S *p, int64_t n) : x(p), V(n) {
        off = int((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(S));
        chunks = uint32_t((n + off + E - 1) / E);
    }
    __device__ __forceinline__ int64_t first_of(uint32_t c) const { return int64_t(c) * E - off; }
    // A chunk as it lies in memory; only whole ones (not the row's first or last) may be asked for.
    __device__ __forceinline__ uint4 whole(uint32_t c) const {
        return __ldcs(reinterpret_cast<const uint4 *>(x + first_of(c)));
    }
    __device__ __forceinline__ bool is_whole(uint32_t c) const { return first_of(c) >= 0 && first_of(c) + E <= V; }
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[E]) {
        const S *s = reinterpret_cast<const S *>(&u);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = to_f32<S>(s[e]);
    }
    __device__ __forceinline__ void load(uint32_t c, float (&v)[E]) const {
        if (is_whole(c)) {
            unpack(whole(c), v);
            return;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t i = first_of(c) + e;
            v[e] = i >= 0 && i < V ? to_f32<S>(x[i]) : -INFINITY;
        }
    }
};

// What has been seen: m, l = sum e^(x - m), w = sum e^(x - m) (x - m).
struct Sums {
    float m, l, w;
};
// The same against another maximum.  (Where nothing has been seen l and w are zero, and the
// difference, held above -150, stands for nothing.)
__device__ __forceinline__ Sums moved(Sums a, float to) {
    const float d = fmaxf(a.m - to, -150.0f), f = ex2(d * kLog2e);
    return {to, a.l * f, f * fmaf(a.l, d, a.w)};
}
__device__ __forceinline__ Sums joined(Sums a, Sums b) {
    const float m = max_nan(a.m, b.m);
    a = moved(a, m);
    b = moved(b, m);
    return {m, a.l + b.l, a.w + b.w};
}

template <typename S>
__global__ void __launch_bounds__(kThreads, kCtas)
    logprob_kernel(const __grid_constant__ trit_logprob_job J, uint32_t *err, int cluster) {
    constexpr int E = Row<S>::E;
    __shared__ u64 keys[kRoom];
    __shared__ u64 tops[kMaxCluster][TRIT_MAX_TOP];     // in the first CTA: every CTA's top entries
    __shared__ Sums sums[kMaxCluster];                  // and sums
    __shared__ Sums warp_sums[kWarps];
    __shared__ u64 groups[kGroups];
    __shared__ uint16_t who[kThreads];
    __shared__ u64 sh_bound, sh_last;
    __shared__ int sh_found, sh_who;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t r = blockIdx.x / cluster;
    const int rank = int(blockIdx.x - r * cluster), N = J.top_n;
    // the first CTA's shared memory may be written once it is known to run: arrive here, wait before the store
    if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");
    pdl_wait();
    pdl_launch();
    const Row<S> row(static_cast<const S *>(J.logits) + r * J.stride, J.V);
    const uint32_t from = uint32_t(u64(row.chunks) * rank / cluster), to = uint32_t(u64(row.chunks) * (rank + 1) / cluster);
    if (tid == 0) {
        sh_found = 0;
        sh_who = 0;
    }
    int token = -1;
    float given = 0.0f;
    if (tid == 0 && rank == 0 && J.tokens) {
        token = J.tokens[r];
        if (token >= 0 && token < J.V) given = to_f32<S>(row.x[token]);
    }

    float m = -INFINITY;
    u64 l2[2] = {0, 0}, w2[2] = {0, 0};        // l and w in four parts
    uint32_t top_chunk = 0;
    auto raised = [&](float cm, uint32_t c) {
        if (!(cm <= m)) {
            const float to = max_nan(m, cm);      // once NaN, always
            const float d = fmaxf(m - to, -150.0f), f = ex2(d * kLog2e);
            const u64 dd = pack2(d, d), ff = pack2(f, f);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                w2[k] = mul2(ff, fma2(l2[k], dd, w2[k]));
                l2[k] = mul2(ff, l2[k]);
            }
            m = to;
            top_chunk = c;
        }
        return m != -INFINITY;
    };
    auto add = [&](float2 x, int k) {
        float2 d = unpack2(add2(pack2(x.x, x.y), pack2(-m, -m)));
        d.x = fmaxf(d.x, -150.0f);            // -inf: e^d is 0, and 0 d must not be NaN
        d.y = fmaxf(d.y, -150.0f);
        const u64 dd = pack2(d.x, d.y);
        const float2 t = unpack2(mul2(dd, pack2(kLog2e, kLog2e)));
        const u64 e = pack2(ex2(t.x), ex2(t.y));
        l2[k] = add2(l2[k], e);
        w2[k] = fma2(e, dd, w2[k]);
    };
    auto see_whole = [&](uint4 u, uint32_t c) {
        if (!raised(greatest<S>(u), c)) return;
        if constexpr (sizeof(S) == 4) {
            add(make_float2(__uint_as_float(u.x), __uint_as_float(u.y)), 0);
            add(make_float2(__uint_as_float(u.z), __uint_as_float(u.w)), 1);
        } else {
            add(unpack16<S>(u.x), 0);
            add(unpack16<S>(u.y), 1);
            add(unpack16<S>(u.z), 0);
            add(unpack16<S>(u.w), 1);
        }
    };
    auto see = [&](uint32_t c) {              // a chunk that may reach out of the row
        float v[E], cm = -INFINITY;
        row.load(c, v);
#pragma unroll
        for (int e = 0; e < E; ++e) cm = max_nan(cm, v[e]);
        if (!raised(cm, c)) return;
#pragma unroll
        for (int e = 0; e < E; e += 2) add(make_float2(v[e], v[e + 1]), (e >> 1) & 1);
    };
    uint32_t c = from + tid;
    // the row's first chunk if it is not whole; whole chunks, kFlight at a time; what is left one by one
    if (c < to && !row.is_whole(c)) {
        see(c);
        c += kThreads;
    }
    const uint32_t whole = from < to && !row.is_whole(to - 1) ? to - 1 : to;
    // (the next kFlight are asked for before these are looked at)
    uint4 u[kFlight];
    bool more = c + (kFlight - 1) * kThreads < whole;
    if (more) {
#pragma unroll
        for (int k = 0; k < kFlight; ++k) u[k] = row.whole(c + k * kThreads);
    }
    while (more) {
        uint4 now[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) now[k] = u[k];
        const uint32_t next = c + kFlight * kThreads;
        more = next + (kFlight - 1) * kThreads < whole;
        if (more) {
#pragma unroll
            for (int k = 0; k < kFlight; ++k) u[k] = row.whole(next + k * kThreads);
        }
#pragma unroll
        for (int k = 0; k < kFlight; ++k) see_whole(now[k], c + k * kThreads);
        c = next;
    }
    for (; c < to; c += kThreads) see(c);
    const float2 la = unpack2(add2(l2[0], l2[1])), wa = unpack2(add2(w2[0], w2[1]));
    Sums a = {m, la.x + la.y, wa.x + wa.y};

    const u64 best = N && a.m > -INFINITY ? key_of(a.m, top_chunk) : 0;      // (a NaN row's keys are not used)
    // the sums of the CTA
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const Sums b = {__shfl_xor_sync(~0u, a.m, o), __shfl_xor_sync(~0u, a.l, o), __shfl_xor_sync(~0u, a.w, o)};
        a = joined(a, b);
    }
    if (lane == 0) warp_sums[warp] = a;
    if (N) {
        u64 g = best;
#pragma unroll
        for (int o = kThreads / kGroups / 2; o; o >>= 1) {
            const u64 x = __shfl_xor_sync(~0u, g, o);
            g = x > g ? x : g;
        }
        if (tid % (kThreads / kGroups) == 0) groups[tid / (kThreads / kGroups)] = g;
    }
    __syncthreads();
    a = lane < kWarps ? warp_sums[lane] : Sums{-INFINITY, 0.0f, 0.0f};
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) {
        const Sums b = {__shfl_xor_sync(~0u, a.m, o), __shfl_xor_sync(~0u, a.l, o), __shfl_xor_sync(~0u, a.w, o)};
        a = joined(a, b);
    }
    a = {__shfl_sync(~0u, a.m, 0), __shfl_sync(~0u, a.l, 0), __shfl_sync(~0u, a.w, 0)};
    const bool fine = a.m < INFINITY;          // neither NaN nor +inf in this CTA's part

    int found = 0;
    if (N && fine) {
        // the bound: the N-th greatest of the groups
        if (tid < kGroups) {
            const u64 g = groups[tid];
            int above = 0;
#pragma unroll 8
            for (int i = 0; i < kGroups; ++i) above += groups[i] > g || (groups[i] == g && i < tid);
            if (above == N - 1) sh_bound = g;
        }
        __syncthreads();
        const u64 bound = sh_bound ? sh_bound : 1;
        if (best >= bound) who[atomicAdd(&sh_who, 1)] = uint16_t(tid);
        __syncthreads();
        const int n = sh_who;
        for (int i = warp; i < n; i += kWarps) {
            const int64_t stride = int64_t(32) * kThreads;
            for (int64_t k = int64_t(from) + who[i] + int64_t(lane) * kThreads; k < to; k += stride) {
                float v[E];
                row.load(uint32_t(k), v);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (key_of(v[e], uint32_t(k)) >= bound) {
                        const int at = atomicAdd(&sh_found, 1);
                        if (at < kRoom) keys[at] = key_of(v[e], uint32_t(row.first_of(uint32_t(k)) + e));
                    }
            }
        }
        __syncthreads();
        found = sh_found;
        u64 *mine = tops[rank];       // this CTA's list
        for (int i = tid; i < N; i += kThreads) mine[i] = 0;
        __syncthreads();
        if (found <= kRoom) {
            for (int i = tid; i < found; i += kThreads) {
                const u64 k = keys[i];
                int above = 0;
                for (int j = 0; j < found; ++j) above += keys[j] > k;
                if (above < N) mine[above] = k;
            }
        } else {
            // too many to hold: one entry a pass, the greatest below the one before
            if (tid == 0) sh_last = ~0ull;
            for (int i = 0; i < N; ++i) {
                __syncthreads();
                const u64 last = sh_last;
                u64 k = 0;
                for (uint32_t c1 = from + tid; c1 < to; c1 += kThreads) {
                    float v[E];
                    row.load(c1, v);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const u64 x = key_of(v[e], uint32_t(row.first_of(c1) + e));
                        if (x < last && x > k) k = x;
                    }
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    const u64 x = __shfl_xor_sync(~0u, k, o);
                    k = x > k ? x : k;
                }
                if (lane == 0) groups[warp] = k;
                __syncthreads();
                if (tid == 0) {
                    for (int w = 1; w < kWarps; ++w) k = groups[w] > k ? groups[w] : k;
                    mine[i] = k;
                    sh_last = k;
                }
            }
        }
    }
    __syncthreads();
    if (cluster > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (rank != 0) {
            uint32_t at;
            if (N && fine)
                for (int i = tid; i < N; i += kThreads) {
                    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(uint32_t(__cvta_generic_to_shared(&tops[rank][i]))));
                    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(tops[rank][i]) : "memory");
                }
            if (tid == 0) {
                asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(uint32_t(__cvta_generic_to_shared(&sums[rank]))));
                asm volatile("st.shared::cluster.f32 [%0], %1;\n st.shared::cluster.f32 [%0+4], %2;\n st.shared::cluster.f32 [%0+8], %3;" ::"r"(at),
                             "f"(a.m), "f"(a.l), "f"(a.w)
                             : "memory");
            }
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank != 0) return;
        for (int i = 1; i < cluster; ++i) a = joined(a, sums[i]);
    }
    const bool good = a.m < INFINITY, empty = a.m == -INFINITY;
    const float nan = __int_as_float(0x7fffffff);
    const float log_l = logf(a.l);             // l >= 1 of a row with a token
    if (tid == 0) {
        if (empty) raise_flag(err, TRIT_ERR_EMPTY);
        if (J.logprob) {
            float v = !good ? nan : empty ? -INFINITY : (given - a.m) - log_l;
            if (token == -1) v = 0.0f;
            else if (token < 0 || token >= J.V) {
                raise_flag(err, TRIT_ERR_INDEX);
                v = -INFINITY;
            }
            J.logprob[r] = v;
        }
        if (J.entropy) J.entropy[r] = !good ? nan : empty ? 0.0f : log_l - a.w / a.l;
    }
    if (!N) return;
    auto put = [&](int at, u64 k) {
        J.top_tokens[r * N + at] = k ? int32_t(0xffffffffu - uint32_t(k)) : -1;
        J.top_logprobs[r * N + at] = k ? (value_of(uint32_t(k >> 32)) - a.m) - log_l : -INFINITY;
    };
    if (!good) {
        for (int i = tid; i < N; i += kThreads) {
            J.top_tokens[r * N + i] = -1;
            J.top_logprobs[r * N + i] = nan;
        }
    } else if (cluster == 1) {
        for (int i = tid; i < N; i += kThreads) put(i, tops[0][i]);
    } else {
        for (int i = tid; i < N * cluster; i += kThreads) {
            const u64 k = tops[i / N][i % N];
            int above = 0;      // zeros (no entry) rank behind all entries, among themselves in this order
            for (int j = 0; j < N * cluster; ++j) {
                const u64 x = tops[j / N][j % N];
                above += x > k || (x == k && j < i);
            }
            if (above < N) put(above, k);
        }
    }
}

template <typename S>
cudaError_t launch(const trit_logprob_job &J, uint32_t *err, cudaStream_t s) {
    // CTAs that share a row: as many as leave every SM two, and each 2048 entries at least
    const int64_t room = 2 * int64_t(device_sm_count());
    int cluster = kMaxCluster;
    while (cluster > 1 && (J.rows * cluster > room || J.V < int64_t(cluster) * 2048)) cluster /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(J.rows * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, logprob_kernel<S>, J, err, cluster);
}

}  // namespace

cudaError_t launch_logprobs(const trit_logprob_job &J, uint32_t *err, cudaStream_t s) {
    return J.dtype == TRIT_F32    ? launch<float>(J, err, s)
           : J.dtype == TRIT_BF16 ? launch<__nv_bfloat16>(J, err, s)
                                  : launch<__half>(J, err, s);
}

}  // namespace trit
