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

#include "trit_attn_items.cuh"

namespace trit {
namespace attn {
namespace {

// Keys of a warp's stage: 8 KB of K and V either way (measured against 16 keys
// for D = 64 too, where a stage's fixed work then outweighs its products).
__host__ __device__ constexpr int keys_of_stage(int D) { return D == 64 ? 32 : 16; }

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

constexpr int kStages = 2;
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
                float k = A.scale2;
                if (far_score(base)) {
#pragma unroll
                    for (int km = 0; km < KM; ++km) {
                        s[km][n][e] = __fmul_rn(s[km][n][e], A.scale2);
                        s[km][n][2 + e] = __fmul_rn(s[km][n][2 + e], A.scale2);
                    }
                    k = 1.0f;
                }
                alpha[n][e] = ex2(m[n][e] - base);
                moved |= alpha[n][e] != 1.0f;
                m[n][e] = top;
                float sum = 0.0f;
#pragma unroll
                for (int km = 0; km < KM; ++km)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float &v = s[km][n][2 * i + e];
                        v = ex2(fmaf(v, k, -base));
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
            if (!direct && J.batch.prefix_len == 0) join_last<T, D, RT>(A, S, p, rows, W, count, scratch);
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

// Dynamic shared memory of a CTA: rings, query tiles, warps' (m, l), the batch.
size_t smem_of(const Args &A) {
    const int D = A.J.cache.head_dim;
    return size_t(kWarps) * kStages * (4 * keys_of_stage(D) * D) + size_t(kStages + 1) * A.RT * D * 2 +
           kWarps * A.RT * 8 + kWarps * 4 + (size_t(A.J.batch.B) * 3 + 1) * 4;
}

Args layout(const trit_attn_job &J) {
    return layout_of(J, kWarps * keys_of_stage(J.cache.head_dim), smem_of, prefix_on_tensor_cores(J));
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
