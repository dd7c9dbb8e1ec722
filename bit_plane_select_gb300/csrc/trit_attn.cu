// trit_attn_paged: out = softmax(scale q K^T) V over a paged cache, the shared
// prefix read once for the batch.
//
// The keys of every item (trit_attn.cuh) are cut into steps of 64 (128 where D = 64), all steps of
// the call are laid end to end and cut into equal chunks, whatever the lengths
// (which only the device knows), one per CTA; beside the prefix kernel of
// trit_attn_prefix.cu, as many as its CTAs leave room for.  A chunk
// may end one item, cover several and begin another.  Items that do not lie in one
// chunk leave partial results, joined by the last of the item's CTAs where
// there is no prefix and by a second launch where there is one (a prefix
// part belongs to many sequences).
//
// Few rows share a key (R = T Hq/Hkv, 4 in a plain decode step), so the cost is
// reading K and V: 4 D bytes a key against 4 D R flops.  A step's keys go 16
// (32 where D = 64) to a warp; every warp has its own ring of two such stages of K and V,
// filled by 16-byte asynchronous copies a stage ahead, so warps never wait
// for one another inside an item.  S^T = K Q^T and O^T += V^T P^T are 16-bit
// mma.sync with fp32 sums, the rows on the n8 side: four rows fill half a tile, not a
// quarter of an m16 one, and O takes D/4 registers per 8 rows.  The rows' m and l
// live in registers and O is only rescaled when a maximum moved.
// P is rounded to the cache's 16-bit type for the second product: relative
// 2^-9 (bf16) or 2^-12 (fp16) of each term on average, the size of the output's own rounding.
// Two sequences of 110500 and 131001 keys of 5 heads of 128, 618 MB: 102 to 104 us, 6.0
// TB/s, 90% of a copy's rate.
#include <type_traits>

#include "trit_attn.cuh"
#include "trit_tc.cuh"

namespace trit {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr size_t kSmemPerSm = 228 * 1024;   // 1 KB of it is taken by every CTA
// Keys of a warp's stage: 8 KB of K and V either way (measured against 16 keys
// for D = 64 too, where a stage's fixed work then outweighs its products).
__host__ __device__ constexpr int keys_of_stage(int D) { return D == 64 ? 32 : 16; }

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
// Whether one of two 16-bit values is an infinity or NaN, and a pair with such values
// replaced by 0.
template <typename T>
__host__ __device__ constexpr uint32_t inf_bits() { return 0x7c00u; }
template <>
__host__ __device__ constexpr uint32_t inf_bits<__nv_bfloat16>() { return 0x7f80u; }
template <typename T>
__device__ __forceinline__ uint32_t finite_pair(uint32_t v) {
    constexpr uint32_t kInf = inf_bits<T>();
    return ((v & 0x7fffu) >= kInf ? 0u : v & 0xffffu) | (((v >> 16) & 0x7fffu) >= kInf ? 0u : v & 0xffff0000u);
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

// A warp's stage of 16 keys: K then V, rows of D 16-bit values whose 16-byte
// chunk c lies at c ^ (row & 7), so that the eight rows of an ldmatrix fall on
// different banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
    return uint32_t(row * D * 2 + ((c ^ (row & 7)) << 4));
}

// The pages of the coming stages' keys, 16 keys by lane, read ahead of their use:
// the table's latency would otherwise stand before every stage's copies.
struct Pages {
    int id;      // lane i: the page of 16-key group i of the warp's stages from `from` on
    int from;
};
template <int D>
__device__ __forceinline__ Pages pages_of(const Args &A, const Keys &K, int step, int warp, int lane) {
    constexpr int KW = keys_of_stage(D), PP = KW / 16;
    Pages P;
    P.from = step;
    const int k = (step + lane / PP) * (KW * kWarps) + warp * KW + (lane % PP) * 16;
    const int col = A.page_shift >= 0 ? k >> A.page_shift : k / A.J.cache.page_size;
    P.id = k >= 0 && k < K.n ? __ldg(K.table + col) : -1;
    return P;
}

// Issues the copies of keys [key0, key0 + KW) of head h.  Rows past the end, and
// rows of pages outside the cache, are filled with zeros.
template <int D>
__device__ __forceinline__ void load_stage(const Args &A, const Keys &K, const Pages &P, int h, int step, int warp,
                                           uint32_t stage, int lane) {
    constexpr int KW = keys_of_stage(D);
    constexpr int CH = D / 8;            // chunks of a row
    constexpr int RI = 32 / CH;          // rows of one copy instruction
    constexpr uint32_t VAT = KW * D * 2;
    const trit_kv_cache &C = A.J.cache;
    const int c = lane % CH, r0 = lane / CH;
    // row r0 + j RI: r0 < RI, so its swizzled chunk is (c ^ r0) ^ (j RI & 7)
    const uint32_t dst = stage + r0 * D * 2, x = uint32_t(c ^ r0) << 4;
    const char *kb = static_cast<const char *>(C.k) + 2 * (h * C.head_stride + c * 8);
    const int64_t to_v = static_cast<const char *>(C.v) - static_cast<const char *>(C.k);
    const int n = K.n, key0 = step * KW * kWarps + warp * KW;
    if ((C.page_size & 15) == 0) {
        constexpr int PJ = 16 / RI;      // copy instructions of 16 keys, which lie in one page
        const int64_t hop = int64_t(RI) * 2 * C.slot_stride;
#pragma unroll
        for (int p = 0; p < KW / 16; ++p) {
            const int k0 = key0 + p * 16;
            const int slot = A.page_shift >= 0 ? k0 & (C.page_size - 1) : k0 % C.page_size;
            const int page = __shfl_sync(~0u, P.id, (step - P.from) * (KW / 16) + p);
            const bool good = page >= 0 && page < C.pages;
            if (!good && k0 < n) raise_flag(A.err, TRIT_ERR_INDEX);
            const int live = good ? n - k0 : 0;          // rows of the 16 that are there
            const char *src = kb + (good ? 2 * (page * C.page_stride + int64_t(slot + r0) * C.slot_stride) : 0);
#pragma unroll
            for (int j = 0; j < PJ; ++j) {
                const int jj = p * PJ + j;
                const uint32_t to = dst + jj * RI * D * 2 + (x ^ uint32_t(((jj * RI) & 7) << 4));
                const bool ok = r0 + j * RI < live;
                const char *at = ok ? src + j * hop : kb;
                cp_async16(to, at, ok);
                cp_async16(to + VAT, at + to_v, ok);
            }
        }
        return;
    }
#pragma unroll 4
    for (int j = 0; j < KW / RI; ++j) {
        const int key = key0 + r0 + j * RI;
        const uint32_t to = dst + j * RI * D * 2 + (x ^ uint32_t(((j * RI) & 7) << 4));
        bool ok = key < n;
        const char *at = kb;
        if (ok) {
            const int col = key / C.page_size;
            const int page = __ldg(K.table + col);
            ok = page >= 0 && page < C.pages;
            if (ok) at += 2 * (page * C.page_stride + int64_t(key - col * C.page_size) * C.slot_stride);
            else raise_flag(A.err, TRIT_ERR_INDEX);
        }
        cp_async16(to, at, ok);
        cp_async16(to + VAT, at + to_v, ok);
    }
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

constexpr int kStages = 2;
// CTAs per SM by the row tiles' registers (shared memory allows three).
__host__ __device__ constexpr int ctas_of(int NB) { return NB <= 2 ? kMostCtas : 2; }

template <typename T, int D, int NB>
__global__ void __launch_bounds__(kThreads, ctas_of(NB)) attn_kernel(const __grid_constant__ Args A) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int RT = 8 * NB;
    constexpr int KW = keys_of_stage(D), kStep = KW * kWarps;
    constexpr int kStageBytes = 2 * KW * D * 2;
    constexpr int kQueries = kStages + 1;     // query tiles: the loads run at most kStages items ahead
    static_assert(kStageBytes >= 16 * D * 4, "a stage holds one m16 tile of fp32 sums");
    const trit_attn_job &J = A.J;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = smem + warp * kStages * kStageBytes;
    const uint32_t ring_at = tc::smem_u32(ring);
    const uint32_t q_at = tc::smem_u32(smem + kWarps * kStages * kStageBytes), q_bytes = RT * D * 2;
    float *stats = reinterpret_cast<float *>(smem + kWarps * kStages * kStageBytes + kQueries * q_bytes);   // [kWarps][RT] (m, l)
    int32_t *scratch = reinterpret_cast<int32_t *>(stats + kWarps * RT * 2);
    Batch S;
    S.cum = scratch + kWarps;
    S.len = S.cum + A.J.batch.B + 1;
    S.fresh = S.len + A.J.batch.B;
    const int32_t *cum = S.cum;

    // after the prefix kernel nothing is left to wait for until the end
    if (!A.tc_items) pdl_wait();
    pdl_launch();
    {   // the page table on its way to L2 while the lengths are: every CTA a few lines of it
        const int64_t ints = int64_t(J.batch.B - 1) * J.batch.table_stride + J.batch.table_pages;
        const int64_t at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 32;
        if (at < ints) asm volatile("prefetch.global.L2 [%0];" ::"l"(J.batch.table + at));
    }
    count_steps<kStep>(A, S, scratch, blockIdx.x == 0);
    const int B = J.batch.B, Hkv = J.cache.heads, G = A.G;
    const int64_t pre = int64_t(Hkv) * A.pre_tiles * A.pre_steps;
    const int64_t W = pre + int64_t(cum[B]) * Hkv * A.own_tiles;
    // this CTA's chunk
    const int64_t count = chunk_count(A, W);
    const int64_t lo = blockIdx.x < count ? chunk_start(blockIdx.x, W, count) : W;
    const int64_t hi = blockIdx.x < count ? chunk_start(blockIdx.x + 1, W, count) : W;

    // the ring runs ahead of the products, across items: keys and values by stage, and
    // an item's queries with its first stage (each warp a quarter of the rows)
    int64_t lu = lo;
    Place lp = {};
    Keys lk = {};
    Pages lpages = {};
    int lq = 0;
    bool lnew = true;
    if (lo < hi) {
        lp = place_of(A, cum, lo);
        lk = keys_of(A, S, lp);
        lpages = pages_of<D>(A, lk, lp.step, warp, lane);
    }
    Place p = lp;
    auto load_queries = [&]() {
        constexpr int CH = D / 8, RI = 32 / CH;
        const int rows = lp.b < 0 ? B * A.R : A.R, c = lane % CH;
#pragma unroll
        for (int j = 0; j < (RT + kWarps * RI - 1) / (kWarps * RI); ++j) {
            const int rl = (j * kWarps + warp) * RI + lane / CH, row = lp.tile * RT + rl;
            if (rl >= RT) continue;
            const int b = lp.b < 0 ? row / A.R : lp.b, r = lp.b < 0 ? row - b * A.R : row;
            const int t = token_of(A, r);
            const bool ok = row < rows && t < S.fresh[b];
            const T *q = static_cast<const T *>(J.q);
            if (ok) q += (int64_t(b) * J.batch.T + t) * J.q_stride + (int64_t(lp.h) * G + r - t * G) * D + c * 8;
            cp_async16(q_at + lq * q_bytes + chunk_at<D>(rl, c), q, ok);
        }
        lq = lq + 1 == kQueries ? 0 : lq + 1;
    };
    auto load_next = [&](int stage) {
        if (lu < hi) {
            if (lnew) {
                load_queries();
                lnew = false;
            }
            load_stage<D>(A, lk, lpages, lp.h, lp.step, warp, ring_at + stage * kStageBytes, lane);
            if (++lu < hi) {
                if (++lp.step == lp.steps) {
                    next_item(A, S, lp);
                    lk = keys_of(A, S, lp);
                    lpages = pages_of<D>(A, lk, 0, warp, lane);
                    lnew = true;
                } else if ((lp.step - lpages.from) * (KW / 16) == 32) {
                    lpages = pages_of<D>(A, lk, lp.step, warp, lane);
                }
            }
        }
        tc::cp_async_commit();
    };
#pragma unroll 1
    for (int s = 0; s < kStages; ++s) load_next(s);

    // the join's copy of the sums, and the rows of sequences without a key (in no CTA's share)
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i <= B; i += kThreads) A.cum[i] = cum[i];
    if (J.batch.prefix_len == 0) {
        for (int b = blockIdx.x; b < B; b += gridDim.x) {
            if (cum[b] != cum[b + 1]) continue;
            const int64_t at = int64_t(b) * J.batch.T * J.q_heads;
            const int64_t rows = int64_t(J.batch.T) * J.q_heads;      // times D: more than 31 bits
            for (int64_t i = threadIdx.x; i < rows * (D / 4); i += kThreads)
                store_out<T>(J, at * D + i * 4, make_float4(0.f, 0.f, 0.f, 0.f));
            for (int64_t i = threadIdx.x; J.lse && i < rows; i += kThreads) J.lse[at + i] = -INFINITY;
        }
    }
    if (lo >= hi) {
        if (A.tc_items && blockIdx.x == 0) pdl_wait();     // see the end
        return;
    }

    // Without a prefix, the last of an item's CTAs to get here joins its parts and leaves
    // the item's counter at zero.  The counter is that of the item's first chunk: no other
    // item begins there and ends elsewhere.
    auto join_last = [&](const Place &q, int rows) {
        const int64_t s0 = int64_t(cum[q.b]) * Hkv * A.own_tiles + (int64_t(q.h) * A.own_tiles + q.tile) * q.steps;
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
                const int t = token_of(A, row), g = row - t * G;
                const int64_t at = (int64_t(q.b) * J.batch.T + t) * J.q_heads + int64_t(q.h) * G + g;
                store_out<T>(J, at * D + c, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                if (J.lse && c == 0) J.lse[at] = lse_of(m, l);
            }
        }
        __syncthreads();   // scratch[0] is free again
    };

    float o[D / 16][NB][4];
    float m[NB][2], l[NB][2];
    int lim[NB][2];
    uint32_t blind = 0;      // the thread's rows that see none of the item's keys
    int nkeys = 0, tiles = 1, first_step = 0, clear = 0;   // no limit lies below `clear`
    uint32_t q_now = 0;                                    // the item's queries
    int cq = 0;

    // A stage that some rows see in part only: an infinity or NaN of V must not reach the rows that
    // its key is hidden from, and their P = 0 would not keep it away (0 * inf is NaN).  Such
    // values are added to the rows that do see them one by one, and are 0 in the stage from
    // there on.  Looking for them costs eight 16-byte reads a lane in those stages alone (none in
    // a step of one token per sequence; 24 sequences of 1 to 5 drafts 40.4 -> 41.5 us).
    auto hide_nonfinite = [&](auto nm, uint8_t *v, int key0, const auto &pf) {
        constexpr int NM = decltype(nm)::value;
        uint4 *v16 = reinterpret_cast<uint4 *>(v);
        constexpr int kPerLane = KW * D / 8 / 32;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const uint4 x = v16[i * 32 + lane];
            const uint32_t top = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                          __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
            bad |= (top & 0xffffu) >= inf_bits<T>() || (top >> 16) >= inf_bits<T>();
        }
        if (!__any_sync(~0u, bad)) return;
#pragma unroll 1
        for (int k = 0; k < KW; ++k) {
            float p[NM][2];       // of this key and the thread's rows 2 (lane % 4) + e
#pragma unroll
            for (int n = 0; n < NM; ++n) {
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < KW / 8; ++i)
                    w |= pf[i >> 1][n][i & 1] & (k >> 3 == i ? ~0u : 0u);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 two = unpack16<T>(__shfl_sync(~0u, w, (2 * (lane & 3) + e) * 4 + ((k & 7) >> 1)));
                    p[n][e] = k & 1 ? two.y : two.x;
                }
            }
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t x = *reinterpret_cast<const uint16_t *>(v + chunk_at<D>(k, 2 * d + i) + 2 * (lane >> 2));
                    if ((x & 0x7fffu) < inf_bits<T>()) continue;
#pragma unroll
                    for (int n = 0; n < NM; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (key0 + k < lim[n][e]) o[d][n][2 * i + e] += p[n][e] * unpack16<T>(x).x;
                }
        }
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < kPerLane; ++i) {
            uint4 x = v16[i * 32 + lane];
            x.x = finite_pair<T>(x.x); x.y = finite_pair<T>(x.y);
            x.z = finite_pair<T>(x.z); x.w = finite_pair<T>(x.w);
            v16[i * 32 + lane] = x;
        }
        __syncwarp();
    };

    // The products of one stage with the item's first NM tiles of 8 rows.  Keys and
    // columns of V are the m16 side, rows the n8 side: S^T = K Q^T, O^T += V^T P^T.  A
    // thread's scores are those of rows 2 (lane % 4) + e, keys lane / 4 and + 8 of a
    // tile; P^T becomes an operand by transposing its 8 x 8 blocks.
    auto products = [&](auto nm, uint32_t kaddr, int key0) {
        constexpr int NM = decltype(nm)::value, KM = KW / 16;
        const uint32_t vaddr = kaddr + KW * D * 2;
        float s[KM][NM][4];
#pragma unroll
        for (int km = 0; km < KM; ++km)
#pragma unroll
            for (int n = 0; n < NM; ++n) s[km][n][0] = s[km][n][1] = s[km][n][2] = s[km][n][3] = 0.0f;
        const int arow = ((lane >> 3) & 1) * 8 + (lane & 7), ach = lane >> 4;
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {     // two k16 steps
            uint32_t qf[2][(NM + 1) / 2 * 2][2];
            if (NM == 1) {
                uint32_t f[4];
                ldsm4(f, q_now + chunk_at<D>(lane & 7, 4 * k2 + (lane >> 3)));
                qf[0][0][0] = f[0]; qf[0][0][1] = f[1]; qf[1][0][0] = f[2]; qf[1][0][1] = f[3];
            } else {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int n2 = 0; n2 < (NM + 1) / 2; ++n2) {
                        uint32_t f[4];
                        ldsm4(f, q_now + chunk_at<D>(n2 * 16 + (lane >> 4) * 8 + (lane & 7),
                                                     2 * (2 * k2 + kk) + ((lane >> 3) & 1)));
                        qf[kk][2 * n2][0] = f[0]; qf[kk][2 * n2][1] = f[1];
                        qf[kk][2 * n2 + 1][0] = f[2]; qf[kk][2 * n2 + 1][1] = f[3];
                    }
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int km = 0; km < KM; ++km) {
                    uint32_t kf[4];
                    ldsm4(kf, kaddr + chunk_at<D>(km * 16 + arow, 2 * (2 * k2 + kk) + ach));
#pragma unroll
                    for (int n = 0; n < NM; ++n) mma16816<T>(s[km][n], kf, qf[kk][n][0], qf[kk][n][1]);
                }
        }
        if (A.flip | ~A.keep) {      // a scale that is not positive
#pragma unroll
            for (int km = 0; km < KM; ++km)
#pragma unroll
                for (int n = 0; n < NM; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[km][n][e] = __uint_as_float((__float_as_uint(s[km][n][e]) & A.keep) ^ (A.flip & 0x80000000u));
        }
        uint32_t pf[KM][NM][2];
        const bool masked = key0 + KW > clear;
        float alpha[NM][2];
        bool moved = false;
#pragma unroll
        for (int n = 0; n < NM; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (masked) {
#pragma unroll
                    for (int km = 0; km < KM; ++km)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (key0 + km * 16 + i * 8 + (lane >> 2) >= lim[n][e]) s[km][n][2 * i + e] = -INFINITY;
                }
                float mx = fmaxf(s[0][n][e], s[0][n][2 + e]);
#pragma unroll
                for (int km = 1; km < KM; ++km) mx = max3(mx, s[km][n][e], s[km][n][2 + e]);
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
                const float top = fmaxf(m[n][e], mx * A.scale2), base = base_of(top);
                alpha[n][e] = ex2(m[n][e] - base);
                moved |= alpha[n][e] != 1.0f;
                m[n][e] = top;
                float sum = 0.0f;
#pragma unroll
                for (int km = 0; km < KM; ++km)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float &v = s[km][n][2 * i + e];
                        v = ex2(fmaf(v, A.scale2, -base));
                        sum += v;
                    }
                l[n][e] = l[n][e] * alpha[n][e] + sum;
            }
#pragma unroll
            for (int km = 0; km < KM; ++km)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    pf[km][n][i] = transposed8(pack16<T>(s[km][n][2 * i], s[km][n][2 * i + 1]));
        }
        if (__any_sync(~0u, moved)) {
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
#pragma unroll
                for (int n = 0; n < NM; ++n) {
                    o[d][n][0] *= alpha[n][0];
                    o[d][n][1] *= alpha[n][1];
                    o[d][n][2] *= alpha[n][0];
                    o[d][n][3] *= alpha[n][1];
                }
        }
        if (masked && clear < nkeys)       // (what follows nkeys is zeros)
            hide_nonfinite(nm, ring + (vaddr - ring_at), key0, pf);
        const int vrow = (lane >> 4) * 8 + (lane & 7), vch = (lane >> 3) & 1;
#pragma unroll
        for (int km = 0; km < KM; ++km)
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                uint32_t vf[4];
                ldsm4t(vf, vaddr + chunk_at<D>(km * 16 + vrow, 2 * d + vch));
#pragma unroll
                for (int n = 0; n < NM; ++n) mma16816<T>(o[d][n], vf, pf[km][n][0], pf[km][n][1]);
            }
    };

    int64_t u = lo;
    bool fresh = true;
    int stage = 0;
    while (u < hi) {
        tc::cp_async_wait<kStages - 1>();
        if (fresh) {
            fresh = false;
            if (u != lo) next_item(A, S, p);
            first_step = p.step;
            nkeys = keys_of(A, S, p).n;
            const int rows = p.b < 0 ? B * A.R : A.R;
            tiles = NB == 1 ? 1 : min(NB, (rows - p.tile * RT + 7) >> 3);
            clear = nkeys;
            blind = 0;
            const int fresh_own = p.b < 0 ? 0 : S.fresh[p.b], len_own = p.b < 0 ? 0 : S.len[p.b];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = p.tile * RT + n * 8 + 2 * (lane & 3) + e;
                    m[n][e] = -INFINITY;
                    l[n][e] = 0.0f;
                    // rows that see no key (padding, tokens before own key 0) or are not there
                    // have no limit, so that they ask for no masks: what they sum up is left out
                    int see = 0;
                    if (p.b >= 0) {
                        const int t = token_of(A, row);
                        if (t < fresh_own) see = len_own - fresh_own + t + 1;
                    } else if (row < rows) {
                        const int b = row / A.R;
                        if (token_of(A, row - b * A.R) < S.fresh[b]) see = nkeys;
                    }
                    if (row >= rows || see <= 0) {
                        blind |= 1u << (2 * n + e);
                        see = nkeys;
                    }
                    lim[n][e] = see;
                    clear = min(clear, see);
                }
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
#pragma unroll
                for (int n = 0; n < NB; ++n) o[d][n][0] = o[d][n][1] = o[d][n][2] = o[d][n][3] = 0.0f;
            clear = min(clear, __shfl_xor_sync(~0u, clear, 1));
            clear = min(clear, __shfl_xor_sync(~0u, clear, 2));
            q_now = q_at + cq * q_bytes;
            cq = cq + 1 == kQueries ? 0 : cq + 1;
            __syncthreads();               // the other warps' rows of the queries
        }
        __syncwarp();
        const int key0 = p.step * kStep + warp * KW;
        uint8_t *st = ring + stage * kStageBytes;
        if (key0 < nkeys) {
            const uint32_t kaddr = ring_at + stage * kStageBytes;
            if (NB == 4 && tiles == 3) products(std::integral_constant<int, NB == 4 ? 3 : 1>{}, kaddr, key0);
            else if (NB > 1 && tiles > NB / 2) products(std::integral_constant<int, NB>{}, kaddr, key0);
            else products(std::integral_constant<int, NB == 4 ? 2 : 1>{}, kaddr, key0);
        }
        __syncwarp();   // every lane has read the stage

        if (p.step + 1 == p.steps || u + 1 == hi) {
            // the item's run in this CTA ends: join the four warps through their free stages
            const bool starts = first_step == 0, ends = p.step + 1 == p.steps;
            const bool whole = starts && ends;
            const bool direct = whole && p.b >= 0 && J.batch.prefix_len == 0;
            const int64_t slot = whole ? (p.b < 0 ? slot_prefix(A, p.h, p.tile) : slot_own(A, p.b, p.h, p.tile))
                                       : 2 * int64_t(blockIdx.x) + (starts ? 1 : 0);
            float *part = A.parts + slot * part_floats(RT, D);
            const int rows = p.b < 0 ? B * A.R : A.R;
#pragma unroll
            for (int half = 0; half < (NB + 1) / 2; ++half) {     // 16 rows at a time
                if (half > 0 && tiles <= 2 * half) break;
                float *mine = reinterpret_cast<float *>(st);
#pragma unroll
                for (int n = 2 * half; n < (NB < 2 * half + 2 ? NB : 2 * half + 2); ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = (n - 2 * half) * 8 + 2 * (lane & 3) + e;
                        float sum = l[n][e];
                        sum += __shfl_xor_sync(~0u, sum, 4);
                        sum += __shfl_xor_sync(~0u, sum, 8);
                        sum += __shfl_xor_sync(~0u, sum, 16);
                        if (lane < 4) {
                            const bool none = (blind >> (2 * n + e)) & 1;
                            stats[(warp * RT + half * 16 + r) * 2] = none ? -INFINITY : m[n][e];
                            stats[(warp * RT + half * 16 + r) * 2 + 1] = none ? 0.0f : sum;
                        }
#pragma unroll
                        for (int d = 0; d < D / 16; ++d)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                mine[r * D + ((d * 16 + i * 8 + (lane >> 2)) ^ ((lane & 3) << 3))] = o[d][n][2 * i + e];
                    }
                __syncthreads();
                constexpr int LR = D / 4, RW = 32 / LR;   // lanes of a row, rows of a warp pass
                const float *all = reinterpret_cast<const float *>(smem + stage * kStageBytes);
                for (int r = warp * RW + lane / LR; r < (RT < 16 ? RT : 16); r += kWarps * RW) {
                    const int row = p.tile * RT + half * 16 + r;
                    if (row >= rows) break;
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stats[(w * RT + half * 16 + r) * 2]);
                    const float base = base_of(top);
                    const int c = (lane % LR) * 4, cs = c ^ (((r >> 1) & 3) << 3);
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    float sum = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float2 ml = *reinterpret_cast<const float2 *>(stats + (w * RT + half * 16 + r) * 2);
                        float4 x = *reinterpret_cast<const float4 *>(
                            all + w * kStages * (kStageBytes / 4) + r * D + cs);
                        // as add_part, without a branch that the next warp's loads would wait for
                        const bool none = ml.x == -INFINITY && ml.y == 0.0f;
                        x.x = none ? 0.0f : x.x; x.y = none ? 0.0f : x.y;
                        x.z = none ? 0.0f : x.z; x.w = none ? 0.0f : x.w;
                        const float f = ex2(ml.x - base);
                        v.x += f * x.x; v.y += f * x.y; v.z += f * x.z; v.w += f * x.w;
                        sum += f * ml.y;
                    }
                    if (direct) {
                        const int t = token_of(A, row), g = row - t * G;
                        const int64_t at = (int64_t(p.b) * J.batch.T + t) * J.q_heads + int64_t(p.h) * G + g;
                        const float inv = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
                        store_out<T>(J, at * D + c, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                        if (J.lse && lane % LR == 0) J.lse[at] = lse_of(top, sum);
                    } else {
                        *reinterpret_cast<float4 *>(part + (half * 16 + r) * D + c) = v;
                        if (lane % LR == 0)
                            *reinterpret_cast<float2 *>(part + RT * D + (half * 16 + r) * 2) = make_float2(top, sum);
                    }
                }
                __syncthreads();
            }
            if (!direct && J.batch.prefix_len == 0) join_last(p, rows);
            fresh = true;
        }
        load_next(stage);
        if (++stage == kStages) stage = 0;
        ++p.step;
        ++u;
    }
    tc::cp_async_wait<0>();
    // the join waits for this grid alone and reads the prefix kernel's results too: one CTA
    // ends after that kernel
    if (A.tc_items && blockIdx.x == 0) pdl_wait();
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

// Dynamic shared memory of a CTA: rings, query tiles, warps' (m, l), the batch.
size_t smem_of(const Args &A) {
    const int D = A.J.cache.head_dim;
    return size_t(kWarps) * kStages * (4 * keys_of_stage(D) * D) + size_t(kStages + 1) * A.RT * D * 2 +
           kWarps * A.RT * 8 + kWarps * 4 + (size_t(A.J.batch.B) * 3 + 1) * 4;
}

// The work's layout from the job's sizes; the grid that a call would use.
Args layout(const trit_attn_job &J) {
    Args A = {};
    A.J = J;
    A.G = J.q_heads / J.cache.heads;
    A.R = J.batch.T * A.G;
    const bool on_tc = prefix_on_tensor_cores(J);
    const int64_t pre_rows = J.batch.prefix_len > 0 && !on_tc ? int64_t(J.batch.B) * A.R : 0;
    const int64_t most_rows = pre_rows > A.R ? pre_rows : A.R;
    A.g_inv = A.R < 65536 ? uint32_t(((int64_t(1) << 32) + A.G - 1) / A.G) : 0;
    if (A.G == 1) A.g_inv = 0;
    A.RT = most_rows > 16 ? 32 : most_rows > 8 ? 16 : 8;
    A.own_tiles = (A.R + A.RT - 1) / A.RT;
    A.pre_tiles = int((pre_rows + A.RT - 1) / A.RT);
    const int kStep = kWarps * keys_of_stage(J.cache.head_dim);
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
    if (on_tc) prefix_layout(A, most);     // and the grid, beside it
    return A;
}

// The workspace: a counter per chunk, [B + 1] sums of steps, partial results.  The counters
// alone carry over from call to call, so they have the same place and room in every
// layout and nothing else is written there: jobs of any sizes may use one workspace in turn.
constexpr int64_t kCountBytes = (kSms * kMostCtas * 4 + 255) / 256 * 256;
int64_t head_bytes(const Args &A) { return kCountBytes + ((int64_t(A.J.batch.B) + 1) * 4 + 255) / 256 * 256; }

int64_t part_bytes(const Args &A) {
    const int64_t slots = slot_prefix(A, 0, 0) + int64_t(A.J.cache.heads) * A.pre_tiles;
    return (slots * part_floats(A.RT, A.J.cache.head_dim) * 4 + 255) / 256 * 256;
}

int64_t bytes_of(const Args &A) { return head_bytes(A) + part_bytes(A) + prefix_part_bytes(A); }

template <typename T, int D, int NB>
cudaError_t launch(const Args &A, cudaStream_t s) {
    const size_t smem = smem_of(A);
    const auto kernel = attn_kernel<T, D, NB>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != cudaSuccess) return e;
    // the prefix kernel first: the next one depends on nothing of it and may start beside it
    if (A.tc_items) e = launch_prefix(A, s);
    if (e == cudaSuccess) e = launch_pdl(kernel, dim3(unsigned(A.grid)), dim3(kThreads), smem, s, A);
    if (e != cudaSuccess) return e;
    if (A.J.batch.prefix_len == 0) return cudaSuccess;
    const int64_t joins = int64_t(A.J.batch.B) * A.J.cache.heads * ((A.R + 3) / 4);
    if (joins <= 2 * kSms) return launch_pdl(join_kernel<T, D, 4>, dim3(unsigned(joins)), dim3(4 * D), 0, s, A);
    return launch_pdl(join_kernel<T, D, 1>, dim3(unsigned(joins)), dim3(D), 0, s, A);
}

template <typename T>
cudaError_t launch_t(const Args &A, cudaStream_t s) {
    if (A.J.cache.head_dim == 128)
        return A.RT == 8 ? launch<T, 128, 1>(A, s) : A.RT == 16 ? launch<T, 128, 2>(A, s) : launch<T, 128, 4>(A, s);
    return A.RT == 8 ? launch<T, 64, 1>(A, s) : A.RT == 16 ? launch<T, 64, 2>(A, s) : launch<T, 64, 4>(A, s);
}

}  // namespace
}  // namespace attn

int64_t attn_workspace_bytes(const trit_attn_job &J) { return attn::bytes_of(attn::layout(J)); }

cudaError_t launch_attn_paged(const trit_attn_job &J, uint32_t *err, cudaStream_t s) {
    attn::Args A = attn::layout(J);
    A.err = err;
    // scores are q k |scale| log2(e), with the sign of a negative scale moved into q; a
    // scale of 0 (masked scores of -inf must not meet it) is zeros for q and 1
    A.scale2 = J.scale == 0.0f ? 1.0f : fabsf(J.scale) * 1.4426950408889634f;
    A.flip = J.scale < 0.0f ? 0x80008000u : 0u;
    A.keep = J.scale == 0.0f ? 0u : 0xffffffffu;
    uint8_t *ws = static_cast<uint8_t *>(J.workspace);
    A.count = reinterpret_cast<uint32_t *>(ws);
    A.cum = reinterpret_cast<int32_t *>(ws + attn::kCountBytes);
    A.parts = reinterpret_cast<float *>(ws + attn::head_bytes(A));
    A.tc_parts = A.parts + attn::part_bytes(A) / 4;
    return J.cache.dtype == TRIT_BF16 ? attn::launch_t<__nv_bfloat16>(A, s) : attn::launch_t<__half>(A, s);
}

}  // namespace trit
