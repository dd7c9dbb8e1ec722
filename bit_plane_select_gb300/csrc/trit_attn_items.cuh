// Attention over a paged cache: the items, steps and chunks of a call, shared by the
// kernels that read K and V themselves (trit_attn.cu: 16 bits, trit_attn4.cu: 4 bits),
// and the joining of their partial results.
#pragma once

#include "trit_attn.cuh"
#include "trit_tc.cuh"

namespace trit {
namespace attn {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr size_t kSmemPerSm = 228 * 1024;   // 1 KB of it is taken by every CTA

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// The transpose of an 8 x 8 matrix of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t transposed8(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Where a step of the work lies.
struct Place {
    int b;         // -1: the prefix
    int h, tile;   // key head, row tile
    int step;      // step of the item's keys
    int steps;     // steps of the item
};

__device__ __forceinline__ Place place_of(const Args &A, const int32_t *cum, int64_t u) {
    Place p;
    const int64_t pre = int64_t(A.J.cache.heads) * A.pre_tiles * A.pre_steps;
    if (u < pre) {
        const int64_t item = quot(u, A.pre_steps);
        p.b = -1;
        p.step = int(u - item * A.pre_steps);
        p.steps = A.pre_steps;
        p.h = int(item) / A.pre_tiles;
        p.tile = int(item - int64_t(p.h) * A.pre_tiles);
        return p;
    }
    const int64_t v = u - pre;
    const int items = A.J.cache.heads * A.own_tiles;
    const int at = int(quot(v, items));            // in steps of one item: cum[b] <= at < cum[b + 1]
    int lo = 0, hi = A.J.batch.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= at) lo = mid;
        else hi = mid - 1;
    }
    p.b = lo;
    p.steps = cum[lo + 1] - cum[lo];
    const int64_t rest = v - int64_t(cum[lo]) * items;
    const int item = int(quot(rest, p.steps));
    p.step = int(rest - int64_t(item) * p.steps);
    p.h = item / A.own_tiles;
    p.tile = item - p.h * A.own_tiles;
    return p;
}

// What a CTA keeps of the batch in shared memory.
struct Batch {
    int32_t *cum;     // [B + 1] steps of the sequences before b
    int32_t *len;     // [B] own lengths, clamped
    int32_t *fresh;   // [B] valid new tokens
};

// The place of the step after p's last one.
__device__ __forceinline__ void next_item(const Args &A, const Batch &S, Place &p) {
    p.step = 0;
    const int tiles = p.b < 0 ? A.pre_tiles : A.own_tiles;
    if (++p.tile < tiles) return;
    p.tile = 0;
    if (++p.h < A.J.cache.heads) return;
    p.h = 0;
    do ++p.b;
    while (S.cum[p.b + 1] == S.cum[p.b]);
    p.steps = S.cum[p.b + 1] - S.cum[p.b];
}

// The keys of a place: their page table, and how many its row tile sees: the tiles of a
// long chunk of new tokens read no further than their last token.
struct Keys {
    const int32_t *table;
    int n;
};
__device__ __forceinline__ Keys keys_of(const Args &A, const Batch &S, const Place &p) {
    Keys k;
    if (p.b < 0) {
        k.table = A.J.batch.prefix_table;
        k.n = int(A.J.batch.prefix_len);
    } else {
        k.table = A.J.batch.table + p.b * A.J.batch.table_stride;
        const int last = token_of(A, min((p.tile + 1) * A.RT, A.R) - 1);
        k.n = max(0, min(S.len[p.b], S.len[p.b] - S.fresh[p.b] + last + 1));
    }
    return k;
}

// Exclusive prefix sums of the sequences' steps into cum[0..B] (shared memory).
template <int kStep>
__device__ __forceinline__ void count_steps(const Args &A, const Batch &S, int32_t *scratch, bool report) {
    const int B = A.J.batch.B, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cap = A.J.batch.table_pages * A.J.cache.page_size;
    for (int i = tid; i < B; i += kThreads) {
        const int n = A.J.batch.lens[i], m = batch_new(A.J.batch, i, report ? A.err : nullptr);
        S.len[i] = n < 0 ? 0 : (n > cap ? cap : n);
        S.fresh[i] = m;
        if (report && (n < 0 || n > cap)) raise_flag(A.err, TRIT_ERR_INDEX);
    }
    __syncthreads();
    const int per = (B + kThreads - 1) / kThreads, from = tid * per;
    int sum = 0;
    for (int i = 0; i < per; ++i)
        if (from + i < B) sum += (S.len[from + i] + kStep - 1) / kStep;
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    int before = inc - sum;
    for (int w = 0; w < warp; ++w) before += scratch[w];
    for (int i = 0; i < per; ++i)
        if (from + i < B) {
            S.cum[from + i] = before;
            before += (S.len[from + i] + kStep - 1) / kStep;
            if (from + i == B - 1) S.cum[B] = before;
        }
    __syncthreads();
}

// One part joined to l and v, which are against `base`.  A part without keys
// (m = -inf, l = 0) holds no sums: its o was never written, or is that of a row that
// sees none of the keys, summed up all the same.
__device__ __forceinline__ void add_part(float2 ml, float4 x, float base, float &l, float4 &v) {
    if (ml.x == -INFINITY && ml.y == 0.0f) return;
    const float f = ex2(ml.x - base);
    l += f * ml.y;
    v.x += f * x.x; v.y += f * x.y; v.z += f * x.z; v.w += f * x.w;
}

// CTAs per SM by the row tiles' registers (shared memory allows three).
__host__ __device__ constexpr int ctas_of(int NB) { return NB <= 2 ? kMostCtas : 2; }

// Without a prefix, the last of an item's CTAs to get here joins its parts and leaves
// the item's counter at zero.  The counter is that of the item's first chunk: no other
// item begins there and ends elsewhere.
template <typename T, int D, int RT>
__device__ __forceinline__ void join_last(const Args &A, const Batch &S, const Place &q, int rows, int64_t W,
                                          int64_t count, int32_t *scratch) {
    const int64_t s0 = int64_t(S.cum[q.b]) * A.J.cache.heads * A.own_tiles + (int64_t(q.h) * A.own_tiles + q.tile) * q.steps;
    const int64_t c0 = chunk_of(s0, W, count);
    const int parts = int(chunk_of(s0 + q.steps - 1, W, count) - c0) + 1;
    uint32_t *arrived = A.count + c0;
    if (threadIdx.x == 0) {
        __threadfence();
        const bool last = atomicAdd(arrived, 1u) + 1 == uint32_t(parts);
        if (last) *arrived = 0;
        __threadfence();
        scratch[0] = last;
    }
    __syncthreads();
    if (scratch[0]) {
        constexpr int CH = D / 4;
        for (int i = threadIdx.x; i < RT * CH; i += kThreads) {
            const int r = i / CH, c = (i % CH) * 4, row = q.tile * RT + r;
            if (row >= rows) break;
            float m = -INFINITY, l = 0.0f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            constexpr int U = 8;     // parts in flight
            for (int k0 = 0; k0 < parts; k0 += U) {
                float2 ml[U];
                float4 x[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    ml[k] = make_float2(-INFINITY, 0.0f);
                    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k0 + k < parts) {
                        const float *part =
                            A.parts + (2 * (c0 + k0 + k) + (k0 + k == 0 ? 1 : 0)) * part_floats(RT, D);
                        ml[k] = __ldcg(reinterpret_cast<const float2 *>(part + RT * D + 2 * r));
                        x[k] = __ldcg(reinterpret_cast<const float4 *>(part + r * D + c));
                    }
                }
                float top = m;
#pragma unroll
                for (int k = 0; k < U; ++k) top = fmaxf(top, ml[k].x);
                const float base = base_of(top), f0 = ex2(m - base);
                m = top;
                l *= f0;
                v.x *= f0; v.y *= f0; v.z *= f0; v.w *= f0;
#pragma unroll
                for (int k = 0; k < U; ++k) add_part(ml[k], x[k], base, l, v);
            }
            const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
            const int t = token_of(A, row), g = row - t * A.G;
            const int64_t at = (int64_t(q.b) * A.J.batch.T + t) * A.J.q_heads + int64_t(q.h) * A.G + g;
            store_out<T>(A.J, at * D + c, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
            if (A.J.lse && c == 0) A.J.lse[at] = lse_of(m, l);
        }
    }
    __syncthreads();   // scratch[0] is free again
}

// Joins the partial results of a call with a prefix: four rows of one
// (sequence, key head) per CTA, four columns per thread, rows by lane first so
// that both forms of partial results (by row, and the tensor-core kernel's by
// column group) are read in whole sectors.  The loads' latency is the cost: where
// there are few rows, kJoin = 4 groups of threads take every fourth part, four at
// a time, else one group takes eight at a time.
template <typename T, int D, int kJoin>
__global__ void __launch_bounds__(kJoin *D) join_kernel(const __grid_constant__ Args A) {
    __shared__ float sh[kJoin > 1 ? kJoin - 1 : 1][6][D];
    pdl_wait();
    const trit_attn_job &J = A.J;
    const int Hkv = J.cache.heads, G = A.G, T_ = J.batch.T, RT = A.RT;
    const int per = (A.R + 3) / 4, bh = int(blockIdx.x) / per;
    const int row4 = int(blockIdx.x) - bh * per, b = bh / Hkv, h = bh - b * Hkv;
    const int tid = threadIdx.x % D, part0 = threadIdx.x / D;            // the group's first part
    const int r4 = row4 * 4 + (tid & 3), c = tid >> 2;                    // columns 4c ..
    const int r = r4 < A.R ? r4 : A.R - 1;
    const int t = r / G, g = r - t * G;

    // the own item's parts
    const int c0 = A.cum[b], n = A.cum[b + 1] - c0;
    const int64_t pre = int64_t(Hkv) * A.pre_tiles * A.pre_steps;
    const int64_t W = pre + int64_t(A.cum[J.batch.B]) * Hkv * A.own_tiles;
    const int64_t count = chunk_count(A, W);
    const int tile = r / RT, rl = r - tile * RT;
    int64_t first = 0;
    int own = 0;
    if (n > 0) {
        const int64_t s0 = pre + (int64_t(c0) * Hkv * A.own_tiles) + (int64_t(h) * A.own_tiles + tile) * n;
        first = chunk_of(s0, W, count);
        own = int(chunk_of(s0 + n - 1, W, count) - first) + 1;
    }
    // the prefix's
    const int64_t fr = int64_t(b) * A.R + r;
    int64_t pfirst = 0;
    int prefix = 0, pitem = 0, prl = 0, pstep = 1;
    if (A.tc_items) {
        const int ptile = int(fr) / kTcRows, group = ptile >> 1;
        const bool pair = 2 * group + 1 < A.tc_tiles;
        prl = int(fr - int64_t(ptile) * kTcRows);
        pfirst = int64_t(h * A.tc_groups + group) * A.tc_splits * 2 + (pair ? ptile & 1 : 0);
        pstep = pair ? 2 : 1;
        prefix = pair ? splits_of(A, W) : 2 * splits_of(A, W);
        if (t >= batch_new(J.batch, b)) prefix = 0;        // padding: that kernel does not look
    } else if (A.pre_tiles) {
        pitem = int(fr) / RT;
        prl = int(fr - int64_t(pitem) * RT);
        const int64_t s0 = (int64_t(h) * A.pre_tiles + pitem) * A.pre_steps;
        pfirst = chunk_of(s0, W, count);
        prefix = int(chunk_of(s0 + A.pre_steps - 1, W, count) - pfirst) + 1;
    }
    const int total = own + prefix;
    float m = -INFINITY, l = 0.0f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = kJoin == 1 ? 8 : 4;     // parts in flight
    for (int i0 = part0; i0 < total; i0 += U * kJoin) {
        float2 ml[U];
        float4 x[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            int i = i0 + k * kJoin;
            ml[k] = make_float2(-INFINITY, 0.0f);
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < total) {
                if (i >= own && A.tc_items) {
                    const float *p = A.tc_parts + (pfirst + int64_t(i - own) * pstep) * part_floats(kTcRows, D);
                    ml[k] = *reinterpret_cast<const float2 *>(p + kTcRows * D + 2 * prl);
                    x[k] = *reinterpret_cast<const float4 *>(p + (c * kTcRows + prl) * 4);
                } else {
                    int64_t slot;
                    int at = rl;
                    if (i < own) {
                        slot = own == 1 ? slot_own(A, b, h, tile) : 2 * (first + i) + (i == 0 ? 1 : 0);
                    } else {
                        at = prl;
                        i -= own;
                        slot = prefix == 1 ? slot_prefix(A, h, pitem) : 2 * (pfirst + i) + (i == 0 ? 1 : 0);
                    }
                    const float *p = A.parts + slot * part_floats(RT, D);
                    ml[k] = *reinterpret_cast<const float2 *>(p + RT * D + 2 * at);
                    x[k] = *reinterpret_cast<const float4 *>(p + at * D + c * 4);
                }
            }
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < U; ++k) top = fmaxf(top, ml[k].x);
        const float base = base_of(top), f0 = ex2(m - base);
        m = top;
        l *= f0;
        v.x *= f0; v.y *= f0; v.z *= f0; v.w *= f0;
#pragma unroll
        for (int k = 0; k < U; ++k) add_part(ml[k], x[k], base, l, v);
    }
    if constexpr (kJoin > 1) {
        if (part0) {
            float(*o)[D] = sh[part0 - 1];
            o[0][tid] = m; o[1][tid] = l;
            o[2][tid] = v.x; o[3][tid] = v.y; o[4][tid] = v.z; o[5][tid] = v.w;
        }
        __syncthreads();
        if (part0) return;
        float top = m;
#pragma unroll
        for (int k = 0; k < kJoin - 1; ++k) top = fmaxf(top, sh[k][0][tid]);
        const float base = base_of(top), f0 = ex2(m - base);
        m = top;
        l *= f0;
        v.x *= f0; v.y *= f0; v.z *= f0; v.w *= f0;
#pragma unroll
        for (int k = 0; k < kJoin - 1; ++k)
            add_part(make_float2(sh[k][0][tid], sh[k][1][tid]),
                     make_float4(sh[k][2][tid], sh[k][3][tid], sh[k][4][tid], sh[k][5][tid]), base, l, v);
    }
    if (r4 >= A.R) return;
    const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
    const int64_t at = (int64_t(b) * T_ + t) * J.q_heads + int64_t(h) * G + g;
    store_out<T>(J, at * D + c * 4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    if (J.lse && c == 0) J.lse[at] = lse_of(m, l);
}

// The work's layout from the job's sizes; the grid that a call would use.  kStep: keys of
// an own step; smem_of: a CTA's dynamic shared memory; on_tc: the prefix is not among the items.
inline Args layout_of(const trit_attn_job &J, int kStep, size_t (*smem_of)(const Args &), bool on_tc, int most_tile = 32,
                      bool split = false) {
    Args A = {};
    A.J = J;
    A.G = J.q_heads / J.cache.heads;
    A.R = J.batch.T * A.G;
    const int64_t pre_rows = J.batch.prefix_len > 0 && !on_tc ? int64_t(J.batch.B) * A.R : 0;
    const int64_t most_rows = pre_rows > A.R ? pre_rows : A.R;
    A.g_inv = A.R < 65536 ? uint32_t(((int64_t(1) << 32) + A.G - 1) / A.G) : 0;
    if (A.G == 1) A.g_inv = 0;
    A.RT = most_rows > 16 ? most_tile : most_rows > 8 ? 16 : 8;
    A.own_tiles = (A.R + A.RT - 1) / A.RT;
    A.pre_tiles = int((pre_rows + A.RT - 1) / A.RT);
    A.own_step = kStep;
    A.pre_steps = on_tc ? 0 : int((J.batch.prefix_len + kStep - 1) / kStep);
    A.page_shift = -1;
    for (int s = 0; s < 31; ++s)
        if (J.cache.page_size == (1 << s)) A.page_shift = s;
    const int64_t cap = (int64_t(J.batch.table_pages) * J.cache.page_size + kStep - 1) / kStep;
    const int64_t most = int64_t(J.cache.heads) * (int64_t(A.pre_tiles) * A.pre_steps +
                                                   int64_t(J.batch.B) * A.own_tiles * cap);
    int per_sm = int(kSmemPerSm / (smem_of(A) + 1024));   // resident together: no CTA waits for another's end
    if (per_sm > ctas_of(A.RT / 8)) per_sm = ctas_of(A.RT / 8);
    if (per_sm < 1) per_sm = 1;
    const int resident = per_sm;
    const int64_t grid = int64_t(kSms) * per_sm;
    A.grid = int(most < grid ? most : grid);
    A.resident = resident;
    A.split = split;
    if (on_tc) prefix_layout(A, most);     // and the grid, beside it
    return A;
}

// The workspace: a counter per chunk, [B + 1] sums of steps, partial results.  The counters
// alone carry over from call to call, so they have the same place and room in every
// layout and nothing else is written there: jobs of any sizes may use one workspace in turn.
constexpr int64_t kCountBytes = (kSms * kMostCtas * 4 + 255) / 256 * 256;
inline int64_t head_bytes(const Args &A) { return kCountBytes + ((int64_t(A.J.batch.B) + 1) * 4 + 255) / 256 * 256; }

inline int64_t part_bytes(const Args &A) {
    const int64_t slots = slot_prefix(A, 0, 0) + int64_t(A.J.cache.heads) * A.pre_tiles;
    return (slots * part_floats(A.RT, A.J.cache.head_dim) * 4 + 255) / 256 * 256;
}

}  // namespace attn
}  // namespace trit
