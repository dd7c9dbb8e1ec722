// trit_logprobs: of a row x of V logits, with m = max x and l = sum e^(x - m),
//     logprob = x[token] - m - ln l,  entropy = ln l - (sum e^(x - m) (x - m)) / l,
// and the top_n largest x, lower indices first among equals.
//
// One pass: a thread keeps (m, l, w) of what it has seen; when its maximum moves from m to m' they
// become f l and f (w + (m - m') l), f = e^(m - m').  Both terms of the entropy are positive, so
// nothing cancels.
//
// The top entries need no second pass over the row.  A thread's chunks of 16 bytes make groups of
// four, and the groups with the same ordinal lie before those with the next.  Order entries by (value,
// lower index) and, coarser, by (value, lower ordinal): a thread knows its greatest entry in the coarse
// order from the running maximum for nothing, and the top_n-th of 64 such (of a few threads each) is a
// bound that at least top_n entries reach, so an entry below it is none of the answer.  Each thread
// also leaves the greatest value of up to 16 stretches of its groups in shared memory; the few that
// reach the bound -- little more than top_n of 4096 -- are read again, and the few dozen entries found are
// ranked by counting.  (Where more than kRoom are found, which takes values that lie by stride, top_n passes
// find one entry each.)
//
// Bound by reading the logits once, or for few rows by latency: then a cluster of up to
// eight CTAs shares a row, and the first of them joins (m, l, w) and ranks the CTAs'
// own top entries, handed over in its shared memory.
//
// A row's sums would cost more than its bytes if written down plainly: an SM gets 24 bytes a clock, 12
// logits of 16 bits, 2.7 clocks of each scheduler for a pair of warps.  So maxima and the hold against -inf are
// taken two 16-bit values at a time, one test of the maximum serves 32 logits, and a pair of logits costs
// one product (t = x log2 e - base), two exponentials, a sum and a product.  Two groups of a thread are on
// their way to its own 16 bytes of a ring: 128 KB an SM, nothing to wait for but its own copies.
// Measured: 2048 rows of 131,072 bf16 logits, top 20: 99 us, 5.4 TB/s (top 0: 85 us; with a subtraction,
// a hold and a test for each chunk 126 us; three groups ahead 104 us: a smaller part of the L1 is left
// to what is read again).  6 rows of 32,000 fp32 logits: 7.0 us.
#include <type_traits>

#include "trit_serve.cuh"

namespace trit {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 4;                   // an SM
constexpr int kGroupsAhead = 2;            // groups of kFlight chunks of a thread in flight
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = 64;                // at least TRIT_MAX_TOP
constexpr int kMaxCluster = 8;
constexpr int kSegments = 16;               // of a thread's chunks, at most
constexpr int kRoom = 2048;                // entries that may reach the bound
constexpr int kFlight = 4;                 // chunks of a group
constexpr int kRingBytes = kGroupsAhead * kFlight * kThreads * 16;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kFar = 1048576.0f;
static_assert(kRingBytes >= kRoom * 8 + kSegments * kThreads * 2, "the ring holds the entries found");
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

// The greater of each of two 16-bit values (NaN if either is).
template <typename S>
__device__ __forceinline__ uint32_t max16(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (std::is_same<S, __half>::value) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// The greatest of 16 bytes of logits (NaN if one is).
template <typename S>
__device__ __forceinline__ float greatest(uint4 u) {
    if constexpr (sizeof(S) == 4) {
        float d;
        asm("{\n .reg .f32 t;\n max.NaN.f32 t, %1, %2, %3;\n max.NaN.f32 %0, t, %4;\n}"
            : "=f"(d)
            : "f"(__uint_as_float(u.x)), "f"(__uint_as_float(u.y)), "f"(__uint_as_float(u.z)), "f"(__uint_as_float(u.w)));
        return d;
    } else {
        const float2 f = unpack16<S>(max16<S>(max16<S>(u.x, u.y), max16<S>(u.z, u.w)));
        return max_nan(f.x, f.y);
    }
}
// The greatest of a group of chunks (NaN if one is).
template <typename S>
__device__ __forceinline__ float greatest_of(const uint4 (&u)[kFlight]) {
    static_assert(kFlight == 4, "");
    if constexpr (sizeof(S) == 4) {
        return max_nan(max_nan(greatest<S>(u[0]), greatest<S>(u[1])), max_nan(greatest<S>(u[2]), greatest<S>(u[3])));
    } else {
        auto of4 = [&](uint32_t a, uint32_t b, uint32_t c, uint32_t d) { return max16<S>(max16<S>(a, b), max16<S>(c, d)); };
        return greatest<S>(make_uint4(of4(u[0].x, u[1].x, u[2].x, u[3].x), of4(u[0].y, u[1].y, u[2].y, u[3].y),
                                      of4(u[0].z, u[1].z, u[2].z, u[3].z), of4(u[0].w, u[1].w, u[2].w, u[3].w)));
    }
}

// A bound for words of logits: one float, or two equal 16-bit values no greater than the
// float asked for.
template <typename S>
struct Word {
    uint32_t v;
    static __device__ __forceinline__ Word below(float x) {
        if constexpr (sizeof(S) == 4) return {__float_as_uint(x)};
        else if constexpr (std::is_same<S, __half>::value) return {__half_as_ushort(__float2half_rd(x)) * 0x10001u};
        else return {__bfloat16_as_ushort(__float2bfloat16_rd(x)) * 0x10001u};
    }
    __device__ __forceinline__ bool finite() const {
        if constexpr (sizeof(S) == 4) return fabsf(__uint_as_float(v)) < INFINITY;
        else return fabsf(unpack16<S>(v).x) < INFINITY;
    }
    __device__ __forceinline__ uint32_t at_least(uint32_t w) const {
        if constexpr (sizeof(S) == 4) return __float_as_uint(fmaxf(__uint_as_float(w), __uint_as_float(v)));
        else return max16<S>(w, v);
    }
};

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
    // A chunk of no logits: all -inf.
    static __device__ __forceinline__ uint4 nothing() {
        const uint32_t w = sizeof(S) == 4 ? 0xff800000u : std::is_same<S, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
        return make_uint4(w, w, w, w);
    }
    // A chunk that reaches out of the row.
    __device__ __forceinline__ uint4 part(uint32_t c) const {
        uint4 u = nothing();
        S *s = reinterpret_cast<S *>(&u);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t i = first_of(c) + e;
            if (i >= 0 && i < V) s[e] = x[i];
        }
        return u;
    }
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
    extern __shared__ __align__(16) uint8_t ring[];     // every thread its own 16 bytes of each chunk
    // once the logits have been seen: [kRoom] entries found, and the segments to look at again
    u64 *const keys = reinterpret_cast<u64 *>(ring);
    uint16_t *const who = reinterpret_cast<uint16_t *>(ring + kRoom * 8);
    __shared__ u64 tops[kMaxCluster][TRIT_MAX_TOP];     // in the first CTA: every CTA's top entries
    __shared__ Sums sums[kMaxCluster];                  // and sums
    __shared__ Sums warp_sums[kWarps];
    __shared__ u64 groups[kGroups];
    __shared__ float segments[kSegments * kThreads];    // greatest of each thread's segments
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

    // What the thread has seen: m, and l and w (in four parts) against 2^t with t = x log2 e - base.  Where
    // base rounds m log2 e, t of m is not 0 but `off`; above kFar, where that would be much, and where the
    // floor below would be -inf, t is taken as (x - m) log2 e.
    enum { kNothing, kNear, kApart };
    int mode = kNothing;
    float m = -INFINITY, base = 0.0f, off = 0.0f;
    Word<S> floor = {};
    u64 l2[2] = {0, 0}, w2[2] = {0, 0};
    uint32_t top_group = 0;
    auto raise = [&](float to, uint32_t g) {
        to = max_nan(m, to);                      // once NaN, always
        floor = Word<S>::below(to - 150.0f);
        mode = fabsf(to) <= kFar && floor.finite() ? kNear : kApart;
        base = to * kLog2e;
        const float new_off = mode == kNear ? fmaf(to, kLog2e, -base) : 0.0f;
        const float d = fmaxf(fmaf(m - to, kLog2e, new_off - off), -300.0f), f = ex2(d);
        const u64 dd = pack2(d, d), ff = pack2(f, f);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            w2[k] = mul2(ff, fma2(l2[k], dd, w2[k]));
            l2[k] = mul2(ff, l2[k]);
        }
        off = new_off;
        m = to;
        top_group = g;
    };
    auto add = [&](float2 x, int k) {
        float2 d;
        if (mode == kNear) {
            d = unpack2(fma2(pack2(x.x, x.y), pack2(kLog2e, kLog2e), pack2(-base, -base)));
        } else {
            d.x = fmaxf(x.x - m, -150.0f) * kLog2e;
            d.y = fmaxf(x.y - m, -150.0f) * kLog2e;
        }
        const u64 e = pack2(ex2(d.x), ex2(d.y));
        l2[k] = add2(l2[k], e);
        w2[k] = fma2(e, pack2(d.x, d.y), w2[k]);
    };
    auto add_chunk = [&](uint4 u) {
        if (mode == kNear) {       // -inf: e^d is 0, and 0 d must not be NaN; what lies 150 below m is 0 too
            u.x = floor.at_least(u.x);
            u.y = floor.at_least(u.y);
            u.z = floor.at_least(u.z);
            u.w = floor.at_least(u.w);
        }
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
    // The thread's chunks are from + tid + j kThreads, kFlight of them a group; its group g and the other threads'
    // lie before all groups g + 1.  Copies go kGroupsAhead groups ahead, of whole chunks.
    const uint32_t lo = from < to && !row.is_whole(from) ? from + 1 : from;
    const uint32_t hi = from < to && !row.is_whole(to - 1) ? to - 1 : to;
    constexpr uint32_t kStride = kFlight * kThreads;
    const uint32_t n_groups = (to - from + kStride - 1) / kStride;
    // a segment is as many groups as make kSegments or fewer of all
    const uint32_t per_segment = (n_groups + kSegments - 1) / kSegments;
    const uint32_t n_segments = n_groups ? (n_groups + per_segment - 1) / per_segment : 0;
    const uint32_t ring_at = uint32_t(__cvta_generic_to_shared(ring)) + tid * 16;
    uint32_t ahead = from + tid;
    auto load_group = [&](uint32_t at) {
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            if (ahead >= lo && ahead < hi)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + k * kThreads * 16), "l"(row.x + row.first_of(ahead)) : "memory");
            ahead += kThreads;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int g = 0; g < kGroupsAhead; ++g) load_group(ring_at + g * kStride * 16);
    uint32_t at = 0, left = per_segment, s_at = tid;
    float seg = -INFINITY;
    for (uint32_t g = 0, c = from + tid; g < n_groups; ++g, c += kStride) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kGroupsAhead - 1) : "memory");
        uint4 u[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) u[k] = *reinterpret_cast<const uint4 *>(ring + at + tid * 16 + k * kThreads * 16);
        if (c < lo || c + (kFlight - 1) * kThreads >= hi) {
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                const uint32_t i = c + k * kThreads;
                if (i < lo || i >= hi) u[k] = i < to ? row.part(i) : Row<S>::nothing();
            }
        }
        load_group(ring_at + at);
        at = at + kStride * 16 == kRingBytes ? 0 : at + kStride * 16;
        const float most = greatest_of<S>(u);
        if (!(most <= m)) raise(most, g);
        if (mode == kNear) {
#pragma unroll
            for (int k = 0; k < kFlight; ++k) add_chunk(u[k]);
        } else if (mode == kApart) {
#pragma unroll 1
            for (int k = 0; k < kFlight; ++k) add_chunk(k == 0 ? u[0] : k == 1 ? u[1] : k == 2 ? u[2] : u[3]);
        }
        seg = fmaxf(seg, most);
        if (--left == 0 || g + 1 == n_groups) {
            segments[s_at] = seg;
            s_at += kThreads;
            seg = -INFINITY;
            left = per_segment;
        }
    }
    // against m itself, and w in the logits' units
    const float2 la = unpack2(add2(l2[0], l2[1])), wa = unpack2(add2(w2[0], w2[1]));
    const float to_m = ex2(-off), l_seen = la.x + la.y;
    Sums a = {m, l_seen * to_m, to_m * kLn2 * fmaf(-off, l_seen, wa.x + wa.y)};
    if (mode != kNothing) {        // the term of m is 1 and none of w is positive: no rounding makes an entropy negative
        a.l = fmaxf(a.l, 1.0f);
        a.w = fminf(a.w, 0.0f);
    }

    const u64 best = N && m > -INFINITY ? key_of(m, top_group) : 0;      // (a NaN row's keys are not used)
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
        // the segments that may hold an entry that reaches it, then those entries
        for (uint32_t g = 0; g < n_segments; ++g)
            if (key_of(segments[g * kThreads + tid], g * per_segment) >= bound)
                who[atomicAdd(&sh_who, 1)] = uint16_t(g * kThreads + tid);
        __syncthreads();
        const uint32_t per = per_segment * kFlight, all = uint32_t(sh_who) * per;
        for (uint32_t p = tid; p < all; p += kThreads) {
            const uint32_t i = p / per, w = who[i], j = w / kThreads * per + p - i * per;
            const uint32_t c = from + w % kThreads + j * kThreads;
            if (c >= to) continue;
            float v[E];
            row.load(c, v);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (key_of(v[e], j / kFlight) >= bound) {
                    const int f = atomicAdd(&sh_found, 1);
                    if (f < kRoom) keys[f] = key_of(v[e], uint32_t(row.first_of(c) + e));
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
    cfg.dynamicSmemBytes = kRingBytes;
    const cudaError_t e = cudaFuncSetAttribute(logprob_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, logprob_kernel<S>, J, err, cluster);
}

}  // namespace

cudaError_t launch_logprobs(const trit_logprob_job &J, uint32_t *err, cudaStream_t s) {
    return J.dtype == TRIT_F32    ? launch<float>(J, err, s)
           : J.dtype == TRIT_BF16 ? launch<__nv_bfloat16>(J, err, s)
                                  : launch<__half>(J, err, s);
}

}  // namespace trit
