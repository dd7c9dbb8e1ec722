// trit_attn_paged4: out = softmax(scale q K^T) V over a paged cache held in 4 bits.
//
// Items, steps, chunks and joins are those of trit_attn_items.cuh: the keys of every
// (sequence, key head, row tile), and of the shared prefix, in steps of 128, all steps of
// the call cut into equal chunks, one per CTA.
//
// A key and head is D codes of 4 bits and D/64 pairs (s, z) for K and as much for V: 144 bytes
// where 16 bits have 512.  At a copy's rate an SM gets 23 of them a clock, 47 codes, so
// turning a code into an operand may cost well under two instructions.  It costs 0.6: with the
// fp16 bit pattern of c as it stands -- c 2^-24, a subnormal -- a word of eight codes is four
// operand registers by masking, the codes of the upper halves of bytes 16 times as large:
//     w & 0x000f000f: c0, c4      w & 0x00f000f0: 16 c1, 16 c5      (w >> 8: c2, c6 and c3, c7).
// K: S^T = K Q^T with the columns of a 32-column chunk in the order that this gives and
// q in the same order, q's odd columns divided by 16.  q is scaled by a power of two per row
// to be large in fp16 (2^14 at its largest column), so that this and fp16's range cost nothing:
// rounding to within 2^-35 of the largest column.  The pairs come in after the products:
//     scale q.k = f sum_groups (s (q'.c) + z sum(q')).
// V: an ldmatrix transposing 16-bit elements, each four columns of a key, gives the same
// word with two keys' codes, so O^T += V^T P^T has the rows of its m16 tiles in the
// order 4 g + i.  p is rounded to fp16 once for all groups (2^15 times as large, so that small ones keep
// their bits); a group's s goes to a copy of it, as s in a unit that fits it, and that
// product is rounded once more: 2 2^-11 of a term s c, or 2^-32 of s c where the weight is small.  One unit, a power of
// two, does for keys whose s lie within 2^8 of one another; others are gone through apart, so that what
// one key's values are off by does not depend on another's (64 sequences of 6000 to 16000 keys of a usual
// spread: 109 us, 110 with one unit for all: a vote a stage).  The z are
// the A operand of one product more, whose row g is group g: sums p z in fp32, 2^-11 of a term.
//
// A warp has its own ring of three stages of 32 keys, so that 165 KB an SM are in flight.  Where pages hold
// runs of 32 keys a stage is copied from one place, else key by key (the address work of that
// was 7% of the time of 64 sequences).  Of two dozen parts and more of a long item the last CTA
// to come has as many on their way as its free stages hold.
//
// A shared prefix that some hundred rows read is written out in 16 bits instead and goes through the
// tensor cores' kernel (prefix_written_out).
//
// Measured, 20 query heads over 5 of 128: 64 sequences of 6000 to 16000 keys 109 us, 4.7 TB/s; two of
// 90000 and 131001 keys 48 us; one of 700 keys 8.6 us.  24 x 5 drafts of 24 heads over 8 of
// 64 behind 8005 keys: 54 us (71 without the tensor cores).  No unit is full (issue 0.54 a clock and scheduler, ALU 53%,
// memory 57%): with 165 registers there are 2.7 warps a scheduler, and an instruction is most often held by the one
// before it in its warp (1.4 warps an issue wait so, 0.55 for the ALU), a third of them masks and shifts.
// Slower: codes by TMA (boxes of 32 keys of 64 bytes: 127 us), four CTAs
// of two stages (registers spill), chunks of uneven length for CTAs of uneven speed (125 us: calls that
// follow one another overlap worse), tiles of 32 rows (2 x 8 drafts over
// 3443 keys 37 us where tiles of 16 take 29: more registers spill and the join has more to do alone).
// Tiles of 16 rows spill too where D = 128 (212 bytes stored, 176 loaded a thread; none in the other forms).
#include <type_traits>

#include "trit_attn_items.cuh"

namespace trit {
namespace attn {
namespace {

constexpr int kStages = 3;
constexpr int KW = 32;                     // keys of a warp's stage
constexpr int kStep = KW * kWarps;
constexpr int kGroup = TRIT_KV4_GROUP;
constexpr float kLift = 15.0f;             // weights are up to 2^15, so that fp16 holds small ones too

template <int D>
struct Shape {
    static constexpr int P = D / kGroup;               // groups of a vector
    static constexpr int CB = D / 2, SB = 4 * P;       // bytes of its codes and pairs
    static constexpr int CH = CB / 16;                 // 16-byte chunks of its codes
    static constexpr int kVAt = KW * CB;               // a stage: K's codes, V's, K's pairs, V's
    static constexpr int kKsAt = 2 * KW * CB, kVsAt = kKsAt + KW * SB;
    static constexpr int kStageBytes = kVsAt + KW * SB;
    static_assert(kStageBytes >= 8 * D * 4, "a stage holds one tile of fp32 sums");
};

struct Args4 {
    Args A;                          // its cache: the codes, strides in vectors
    const uint8_t *k_scale, *v_scale;
    float scale2;                    // scale log2(e)
    int32_t runs;                    // whether 32 keys from a multiple of 32 on always lie side by side
};

__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, bool ok, std::integral_constant<int, 8>) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8u : 0u) : "memory");
}
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, bool ok, std::integral_constant<int, 4>) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4u : 0u) : "memory");
}

// Byte offset of 16-byte chunk c of row r of a tile of codes: eight rows at one c fall on
// eight different quarters of the banks.
template <int D>
__device__ __forceinline__ uint32_t codes_at(int r, int c) {
    return D == 128 ? uint32_t(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)) : uint32_t(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
}
// A query tile as it is loaded.
template <int D>
__device__ __forceinline__ uint32_t query_at(int row, int c) {
    return uint32_t(row * D * 2 + ((c ^ (row & 7)) << 4));
}

// The operand registers of codes 0..3 of each 16 bits.
__device__ __forceinline__ void operands(const uint32_t (&f)[4], int i, uint32_t (&a)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = (i < 2 ? f[j] : f[j] >> 8) & (i & 1 ? 0x00f000f0u : 0x000f000fu);
}
// The same product with nothing before it.
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t mul16(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t half_power2(int e) {       // a pair of 2^e, e in -24..15
    const uint32_t h = e >= -14 ? uint32_t(e + 15) << 10 : 1u << (e + 24);
    return h | h << 16;
}
__device__ __forceinline__ bool odd16(uint32_t pair) {         // an infinity or NaN among two fp16 values
    return (pair & 0x7c00u) == 0x7c00u || (pair & 0x7c000000u) == 0x7c000000u;
}
// What the weights of a row with greatest score x are taken against, so that they are up to 2^kLift.  From 2^24 on
// x less kLift may be no fp32 number: rounded upwards, since a weight of 2^16 is past fp16's range.
__device__ __forceinline__ float lifted(float x) { return __fsub_ru(x, kLift); }
__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }   // e in -126..127

// The same as join_last, but up to `room` parts of a row on their way at once, into a warp's slots of 512 bytes
// (a thread's own 16, so that no other thread waits for them).  Two sequences of 90000 and
// 131001 keys, 46 parts an item: 52.4 us with eight in registers, 48.3 so.
template <typename T, int D, int RT>
__device__ __forceinline__ void join_apart(const Args &A, const Batch &S, const Place &q, int rows, int64_t W,
                                           int64_t count, int32_t *scratch, const uint8_t *slots, int room) {
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
        constexpr int LR = D / 4;                  // lanes of a row
        const int lane = threadIdx.x & 31, j = lane % LR;
        const uint8_t *mine = slots + lane * 16;
        const uint32_t mine_at = tc::smem_u32(mine);
        if (room > LR) room = LR;
        for (int r = threadIdx.x / LR; r - lane / LR < RT; r += kThreads / LR) {      // (a warp's rows together)
            const int row = q.tile * RT + r;
            if (row - lane / LR >= rows) break;
            const bool there = row < rows;
            float m = -INFINITY, l = 0.0f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < parts; k0 += room) {
                const int n = min(room, parts - k0);
                // chunk c's part: at 2 c, or 2 c + 1 where the item begins in it
                const float *first = A.parts + 2 * (c0 + k0) * part_floats(RT, D);
                for (int k = 0; k < n; ++k)
                    cp_async16(mine_at + k * 512, first + (2 * k + (k0 + k == 0 ? 1 : 0)) * part_floats(RT, D) + r * D + j * 4, there);
                tc::cp_async_commit();
                float2 ml = make_float2(-INFINITY, 0.0f);
                if (there && j < n)
                    ml = __ldcg(reinterpret_cast<const float2 *>(
                        first + (2 * j + (k0 + j == 0 ? 1 : 0)) * part_floats(RT, D) + RT * D + 2 * r));
                float top = fmaxf(m, ml.x);
#pragma unroll
                for (int o = LR / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                const float base = base_of(top), f0 = ex2(m - base);
                m = top;
                // -1: a part without keys, which holds no sums
                const float f = ml.x == -INFINITY && ml.y == 0.0f ? -1.0f : ex2(ml.x - base);
                float sum = f == -1.0f ? 0.0f : f * ml.y;
#pragma unroll
                for (int o = LR / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                l = l * f0 + sum;
                v.x *= f0; v.y *= f0; v.z *= f0; v.w *= f0;
                tc::cp_async_wait<0>();
                for (int k = 0; k < n; ++k) {
                    const float fk = __shfl_sync(~0u, f, k, LR);
                    const float4 x = *reinterpret_cast<const float4 *>(mine + k * 512);
                    if (fk == -1.0f) continue;
                    v.x += fk * x.x; v.y += fk * x.y; v.z += fk * x.z; v.w += fk * x.w;
                }
            }
            if (!there) continue;
            const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
            const int t = token_of(A, row), g = row - t * A.G;
            const int64_t at = (int64_t(q.b) * A.J.batch.T + t) * A.J.q_heads + int64_t(q.h) * A.G + g;
            store_out<T>(A.J, at * D + j * 4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
            if (A.J.lse && j == 0) A.J.lse[at] = lse_of(m, l);
        }
    }
    __syncthreads();   // scratch[0] is free again
}

template <typename T, int D, int NB>
__global__ void __launch_bounds__(kThreads, ctas_of(NB)) attn4_kernel(const __grid_constant__ Args4 A4) {
    extern __shared__ __align__(128) uint8_t smem[];
    using Sh = Shape<D>;
    constexpr int P = Sh::P, RT = 8 * NB, kStageBytes = Sh::kStageBytes;
    constexpr int kQueries = kStages + 1;     // query tiles: the loads run at most kStages items ahead
    const Args &A = A4.A;
    const trit_attn_job &J = A.J;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = smem + warp * kStages * kStageBytes;
    const uint32_t ring_at = tc::smem_u32(ring);
    uint8_t *queries = smem + kWarps * kStages * kStageBytes;
    const uint32_t q_at = tc::smem_u32(queries), q_bytes = RT * D * 2;
    uint4 *frag = reinterpret_cast<uint4 *>(queries + kQueries * q_bytes);       // [NB][P][2][32]
    float *facs = reinterpret_cast<float *>(frag + NB * P * 64);                 // [RT] factors f
    float *qsum = facs + RT;                                                     // [RT][P] 2^-24 sum(q')
    float *stats = qsum + RT * P;                                                // [kWarps][RT] (m, l)
    int32_t *scratch = reinterpret_cast<int32_t *>(stats + kWarps * RT * 2);
    Batch S;
    S.cum = scratch + kWarps;
    S.len = S.cum + J.batch.B + 1;
    S.fresh = S.len + J.batch.B;
    const int32_t *cum = S.cum;

    // (beside the prefix kernel, which started after all that this one reads was written)
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
    int lq = 0, page = -1;       // page: of the lane's key of the next stage to load
    bool lnew = true;
    auto key_of_lane = [&]() { return lp.step * kStep + warp * KW + lane; };
    auto fetch_page = [&]() {
        const int k = key_of_lane();
        page = k < lk.n ? __ldg(lk.table + (A.page_shift >= 0 ? k >> A.page_shift : k / J.cache.page_size)) : -1;
    };
    if (lo < hi) {
        lp = place_of(A, cum, lo);
        lk = keys_of(A, S, lp);
        fetch_page();
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
            cp_async16(q_at + lq * q_bytes + query_at<D>(rl, c), q, ok);
        }
        lq = lq + 1 == kQueries ? 0 : lq + 1;
    };
    // The copies of the warp's 32 keys of a step; a lane finds one key's place.  Rows past the
    // end and rows of pages outside the cache are filled with zeros.
    auto load_stage = [&](uint32_t st) {
        if (A4.runs && lp.step * kStep + (warp + 1) * KW <= lk.n && page >= 0 && page < J.cache.pages) {
            // all 32 there, in a row: one place for the warp (every lane's page is the same)
            const int k = lp.step * kStep + warp * KW;
            const int64_t vec = page * J.cache.page_stride + (k & (J.cache.page_size - 1)) + lp.h * J.cache.head_stride;
            const uint8_t *kc = static_cast<const uint8_t *>(J.cache.k) + vec * Sh::CB + lane * 16;
            const uint8_t *vc = static_cast<const uint8_t *>(J.cache.v) + vec * Sh::CB + lane * 16;
            cp_async_small(st + Sh::kKsAt + lane * Sh::SB, A4.k_scale + (vec + lane) * Sh::SB, true, std::integral_constant<int, Sh::SB>{});
            cp_async_small(st + Sh::kVsAt + lane * Sh::SB, A4.v_scale + (vec + lane) * Sh::SB, true, std::integral_constant<int, Sh::SB>{});
            // row lane / CH + j 32 / CH: its swizzle depends on j by a constant
            const uint32_t dst = st + codes_at<D>(lane / Sh::CH, lane % Sh::CH);
#pragma unroll
            for (int j = 0; j < Sh::CH; ++j) {
                cp_async16(dst + j * 512, kc + j * 512, true);
                cp_async16(dst + j * 512 + Sh::kVAt, vc + j * 512, true);
            }
            return;
        }
        const int k = key_of_lane();
        const bool in = k < lk.n, good = in && page >= 0 && page < J.cache.pages;
        if (in && !good) raise_flag(A.err, TRIT_ERR_INDEX);
        const int col = A.page_shift >= 0 ? k >> A.page_shift : k / J.cache.page_size;
        const int64_t vec = good ? page * J.cache.page_stride + int64_t(k - col * J.cache.page_size) * J.cache.slot_stride +
                                       lp.h * J.cache.head_stride
                                 : 0;
        cp_async_small(st + Sh::kKsAt + lane * Sh::SB, A4.k_scale + vec * Sh::SB, good, std::integral_constant<int, Sh::SB>{});
        cp_async_small(st + Sh::kVsAt + lane * Sh::SB, A4.v_scale + vec * Sh::SB, good, std::integral_constant<int, Sh::SB>{});
        const uint32_t there = __ballot_sync(~0u, good);
        constexpr int RI = 32 / Sh::CH;                 // keys of one copy instruction
        const int c = lane % Sh::CH;
#pragma unroll
        for (int j = 0; j < KW / RI; ++j) {
            const int r = j * RI + lane / Sh::CH;
            const int64_t at = __shfl_sync(~0u, vec, r) * Sh::CB + c * 16;
            const bool ok = (there >> r) & 1;
            const uint32_t dst = st + codes_at<D>(r, c);
            cp_async16(dst, static_cast<const uint8_t *>(J.cache.k) + at, ok);
            cp_async16(dst + Sh::kVAt, static_cast<const uint8_t *>(J.cache.v) + at, ok);
        }
    };
    auto load_next = [&](int stage) {
        if (lu < hi) {
            if (lnew) {
                load_queries();
                lnew = false;
            }
            load_stage(ring_at + stage * kStageBytes);
            if (++lu < hi) {
                if (++lp.step == lp.steps) {
                    next_item(A, S, lp);
                    lk = keys_of(A, S, lp);
                    lnew = true;
                }
                fetch_page();
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
            const int64_t rows = int64_t(J.batch.T) * J.q_heads;
            for (int64_t i = threadIdx.x; i < rows * (D / 4); i += kThreads)
                store_out<T>(J, at * D + i * 4, make_float4(0.f, 0.f, 0.f, 0.f));
            for (int64_t i = threadIdx.x; J.lse && i < rows; i += kThreads) J.lse[at + i] = -INFINITY;
        }
    }
    if (lo >= hi) {
        if (A.tc_items && blockIdx.x == 0) pdl_wait();     // see the end
        return;
    }

    float o[P][4][NB][4];        // columns 64 p + 32 (e / 2) + 4 (lane / 4) + i, row 2 (lane % 4) + e % 2
    float z[NB][2];              // of lanes 4 pg + t: sum of p z of group pg, row 2 t + e
    float m[NB][2], l[NB][2];    // what the row's weights are against, and their sum
    int lim[NB][2];
    int unit[P];                 // sums of s c are in units of 2^(unit - 14)
    uint32_t blind = 0;      // the thread's rows that see none of the item's keys
    int nkeys = 0, tiles = 1, first_step = 0, clear = 0;   // no limit lies below `clear`
    int cq = 0;
    // one tile's queries stay in registers
    uint4 held[NB == 1 ? P : 1][2];
    float held_sum[NB == 1 ? P : 1][2], held_fac[2];

    // An item's queries as operands: warp n takes tile n.  Lane (g, t) has of row g the
    // columns 64 p + 32 b + 8 t + 0..7; operand i of chunk b is its columns i and i + 4.
    auto prepare_queries = [&](const uint8_t *raw) {
        if (warp >= NB) return;
        const int row = warp * 8 + (lane >> 2), t = lane & 3;
        float v[P][2][8], most = 0.0f;
#pragma unroll
        for (int pg = 0; pg < P; ++pg)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint4 u = *reinterpret_cast<const uint4 *>(raw + query_at<D>(row, 8 * pg + 4 * b + t));
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = unpack16<T>(w[k]);
                    v[pg][b][2 * k] = f.x;
                    v[pg][b][2 * k + 1] = f.y;
                    most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
        most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
        most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
        // the largest column to [2^14, 2^15), as far as the factor back (2^(24 - e)) stays in range
        int e = 14 - ((__float_as_int(most) >> 23) - 127);
        e = e > 100 ? 100 : e < -100 ? -100 : e;
        const float f[2] = {power2(e), power2(e - 4)};
#pragma unroll
        for (int pg = 0; pg < P; ++pg) {
            uint32_t w[8];
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    w[2 * i + b] = pack16<__half>(v[pg][b][i] * f[i & 1], v[pg][b][i + 4] * f[i & 1]);
                    const float2 r = unpack16<__half>(w[2 * i + b]);
                    sum = fmaf(r.x + r.y, i & 1 ? 16.0f : 1.0f, sum);
                }
            frag[((warp * P + pg) * 2) * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
            frag[((warp * P + pg) * 2 + 1) * 32 + lane] = make_uint4(w[4], w[5], w[6], w[7]);
            sum += __shfl_xor_sync(~0u, sum, 1);
            sum += __shfl_xor_sync(~0u, sum, 2);
            if (t == 0) qsum[row * P + pg] = sum * 0x1p-24f;
        }
        if (t == 0) facs[row] = A4.scale2 * power2(24 - e);
    };

    // The products of one stage with the item's first NM tiles of 8 rows.  MASKED: some row does
    // not see all of its keys.
    auto products = [&](auto nm, auto masked, uint8_t *st, uint32_t st_at, int key0) {
        constexpr int NM = decltype(nm)::value, KM = KW / 16;
        constexpr bool MASKED = decltype(masked)::value;
        const int g = lane >> 2, t2 = 2 * (lane & 3);
        float s[KM][NM][4];
        const int arow = ((lane >> 3) & 1) * 8 + (lane & 7), ach = lane >> 4;
#pragma unroll
        for (int km = 0; km < KM; ++km) {
            // the pairs of keys g and g + 8
            uint32_t ks[2][P];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t *at = st + Sh::kKsAt + (km * 16 + 8 * i + g) * Sh::SB;
                if (P == 2) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(at);
                    ks[i][0] = v.x;
                    ks[i][P - 1] = v.y;
                } else {
                    ks[i][0] = *reinterpret_cast<const uint32_t *>(at);
                }
            }
#pragma unroll
            for (int pg = 0; pg < P; ++pg) {
                uint32_t f[4], a[4][4];
                ldsm4(f, st_at + codes_at<D>(km * 16 + arow, 2 * pg + ach));
#pragma unroll
                for (int i = 0; i < 4; ++i) operands(f, i, a[i]);
                const float2 k0 = unpack16<__half>(ks[0][pg]), k1 = unpack16<__half>(ks[1][pg]);
#pragma unroll
                for (int n = 0; n < NM; ++n) {
                    const uint4 q0 = NB == 1 ? held[NB == 1 ? pg : 0][0] : frag[((n * P + pg) * 2) * 32 + lane];
                    const uint4 q1 = NB == 1 ? held[NB == 1 ? pg : 0][1] : frag[((n * P + pg) * 2 + 1) * 32 + lane];
                    float acc[4];
                    mma16816_first(acc, a[0], q0.x, q0.y);
                    mma16816<__half>(acc, a[1], q0.z, q0.w);
                    mma16816<__half>(acc, a[2], q1.x, q1.y);
                    mma16816<__half>(acc, a[3], q1.z, q1.w);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float qs = NB == 1 ? held_sum[NB == 1 ? pg : 0][e] : qsum[(n * 8 + t2 + e) * P + pg];
                        const float z0 = k0.y * qs, z1 = k1.y * qs;
                        s[km][n][e] = fmaf(k0.x, acc[e], pg ? s[km][n][e] + z0 : z0);
                        s[km][n][2 + e] = fmaf(k1.x, acc[2 + e], pg ? s[km][n][2 + e] + z1 : z1);
                    }
                }
            }
        }
        float alpha[NM][2];
        bool moved = false;
#pragma unroll
        for (int n = 0; n < NM; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = NB == 1 ? held_fac[e] : facs[n * 8 + t2 + e];
                float mx = -INFINITY;
#pragma unroll
                for (int km = 0; km < KM; ++km) {
                    float &v0 = s[km][n][e], &v1 = s[km][n][2 + e];
                    v0 *= f;
                    v1 *= f;
                    if (MASKED) {
                        if (key0 + km * 16 + g >= lim[n][e]) v0 = -INFINITY;
                        if (key0 + km * 16 + 8 + g >= lim[n][e]) v1 = -INFINITY;
                    }
                    mx = max3(mx, v0, v1);
                }
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
                const float to = fmaxf(m[n][e], lifted(mx)), base = base_of(to);
                alpha[n][e] = ex2(m[n][e] - base);
                moved |= alpha[n][e] != 1.0f;
                m[n][e] = to;
                float sum = 0.0f;
#pragma unroll
                for (int km = 0; km < KM; ++km)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float &v = s[km][n][2 * i + e];
                        v = ex2(v - base);
                        sum += v;
                    }
                l[n][e] = l[n][e] * alpha[n][e] + sum;
            }
        if (__any_sync(~0u, moved)) {
#pragma unroll
            for (int n = 0; n < NM; ++n) {
                z[n][0] *= alpha[n][0];
                z[n][1] *= alpha[n][1];
#pragma unroll
                for (int pg = 0; pg < P; ++pg)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[pg][i][n][e] *= alpha[n][e & 1];
            }
        }
        // The pairs of V: a lane looks at one key's.  s counts in a unit, 2^(unit - 14), that keeps s over it in
        // [2^-8, 1) (exactly; an s of 0 and a subnormal one may be less), so that a product p s is as
        // exact as p, whatever other keys hold.  Keys that the unit does not fit move it; where a stage's lie
        // too far apart for one it is gone through in parts, a range of eight exponents each.  In a stage that some
        // rows see in part the ranges are fixed ones: a key hidden from a row then has no part in its roundings.
        uint32_t *own = reinterpret_cast<uint32_t *>(st + Sh::kVsAt + lane * Sh::SB);
        uint32_t left = 0;           // ranges still to come
        auto move_unit = [&](int pg, int to) {
            if (to == unit[pg]) return;
            const float f = power2(unit[pg] - to);
            unit[pg] = to;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NM; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[pg][i][n][e] *= f;
        };
        {
            uint32_t pair[P];
            bool bad = false;
#pragma unroll
            for (int pg = 0; pg < P; ++pg) {
                pair[pg] = own[pg];
                bad |= MASKED && odd16(pair[pg]);
            }
            if (MASKED) {
                // A NaN that some row does not see must not meet its P = 0: it goes to the rows that do, one by
                // one, and out of the stage.
                uint32_t which = __ballot_sync(~0u, bad);
                for (uint32_t more = which; more; more &= more - 1) {
                    const int k = __ffs(int(more)) - 1;
#pragma unroll
                    for (int pg = 0; pg < P; ++pg) {
                        const uint32_t v = __shfl_sync(~0u, pair[pg], k);
                        if (!odd16(v) || g != pg) continue;
#pragma unroll
                        for (int n = 0; n < NM; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (key0 + k < lim[n][e]) z[n][e] += unpack16<__half>(v).x - unpack16<__half>(v).x + unpack16<__half>(v).y;
                    }
                }
                if (which) {
#pragma unroll
                    for (int pg = 0; pg < P; ++pg)
                        if (bad) own[pg] = pair[pg] = odd16(pair[pg]) ? 0u : pair[pg];
                    __syncwarp();
                }
            }
            bool fits = !MASKED;
#pragma unroll
            for (int pg = 0; pg < P; ++pg) fits = fits && (pair[pg] & 0x7fffu) - (uint32_t(unit[pg] - 7) << 10) < (8u << 10);
            if (MASKED || !__all_sync(~0u, fits)) {
                uint32_t there[P];           // exponents of the stage's s that are not 0
#pragma unroll
                for (int pg = 0; pg < P; ++pg)
                    there[pg] = __reduce_or_sync(~0u, pair[pg] & 0x7fffu ? 1u << ((pair[pg] >> 10) & 31u) : 0u);
                bool far = MASKED;
#pragma unroll
                for (int pg = 0; pg < P; ++pg) far |= __clz(int(there[pg])) + __ffs(int(there[pg])) <= 24;     // more than 8
                if (!far) {
#pragma unroll
                    for (int pg = 0; pg < P; ++pg)
                        if (there[pg] & ~(0xffu << (unit[pg] - 7)))
                            move_unit(pg, max(7, min(31, (31 - __clz(int(there[pg])) + __ffs(int(there[pg])) + 7) / 2)));
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int pg = 0; pg < P; ++pg) left |= (there[pg] >> (8 * c)) & 0xffu ? 1u << c : 0u;
                    const int c = __ffs(int(left | 16u)) - 1;
                    left &= left - 1;
                    if (c < 4)
#pragma unroll
                        for (int pg = 0; pg < P; ++pg) move_unit(pg, 8 * c + 7);
                    if (left) {      // K's pairs are no longer needed: V's go there, and to their own place part by part
                        __syncwarp();
#pragma unroll
                        for (int pg = 0; pg < P; ++pg) {
                            own[pg - Sh::kVsAt / 4 + Sh::kKsAt / 4] = pair[pg];
                            own[pg] = int(pair[pg] >> 13 & 3u) == c ? pair[pg] : pair[pg] & 0xffff0000u;
                        }
                        __syncwarp();
                    }
                }
            }
        }
        // the weights as an operand, for all groups
        uint32_t w[KM][NM][2];
#pragma unroll
        for (int km = 0; km < KM; ++km)
#pragma unroll
            for (int n = 0; n < NM; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) w[km][n][i] = transposed8(pack16<__half>(s[km][n][2 * i], s[km][n][2 * i + 1]));
        const int vrow = (lane >> 4) * 8 + (lane & 7), vch = (lane >> 3) & 1;
        for (;;) {
            uint32_t inv[P];
#pragma unroll
            for (int pg = 0; pg < P; ++pg) inv[pg] = half_power2(14 - unit[pg]);
#pragma unroll
            for (int km = 0; km < KM; ++km) {
                // the pairs of keys 2t, 2t + 1 and 8 further: s by keys, in units; z as a product's operand whose
                // row pg is the group's
                uint32_t sp[P][2], za[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t *at = st + Sh::kVsAt + (km * 16 + 8 * i + t2) * Sh::SB;
                    if (P == 2) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(at);
                        sp[0][i] = mul16(prmt(v.x, v.z, 0x5410u), inv[0]);
                        sp[P - 1][i] = mul16(prmt(v.y, v.w, 0x5410u), inv[P - 1]);
                        za[2 * i] = prmt(g == 0 ? v.x : v.y, g == 0 ? v.z : v.w, 0x7632u);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2 *>(at);
                        sp[0][i] = mul16(prmt(v.x, v.y, 0x5410u), inv[0]);
                        za[2 * i] = prmt(v.x, v.y, 0x7632u);
                    }
                    if (g >= P) za[2 * i] = 0;
                }
#pragma unroll
                for (int n = 0; n < NM; ++n) {
                    float zc[4] = {z[n][0], z[n][1], 0.0f, 0.0f};
                    mma16816<__half>(zc, za, w[km][n][0], w[km][n][1]);
                    z[n][0] = zc[0];
                    z[n][1] = zc[1];
                }
#pragma unroll
                for (int pg = 0; pg < P; ++pg) {
                    uint32_t f[4];
                    ldsm4t(f, st_at + Sh::kVAt + codes_at<D>(km * 16 + vrow, 2 * pg + vch));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t a[4];
                        operands(f, i, a);
#pragma unroll
                        for (int n = 0; n < NM; ++n)
                            mma16816<__half>(o[pg][i][n], a, mul16(w[km][n][0], sp[pg][0]), mul16(w[km][n][1], sp[pg][1]));
                    }
                }
            }
            if (!left) break;
            const int c = __ffs(int(left)) - 1;
            left &= left - 1;
            __syncwarp();
#pragma unroll
            for (int pg = 0; pg < P; ++pg) {
                const uint32_t v = own[pg - Sh::kVsAt / 4 + Sh::kKsAt / 4];
                own[pg] = int(v >> 13 & 3u) == c ? v & 0xffffu : 0u;      // (z has been added)
                move_unit(pg, 8 * c + 7);
            }
            __syncwarp();
        }
    };
    auto stage_products = [&](auto masked, uint8_t *st, uint32_t st_at, int key0) {
        if (NB > 1 && tiles > 1) products(std::integral_constant<int, NB>{}, masked, st, st_at, key0);
        else products(std::integral_constant<int, 1>{}, masked, st, st_at, key0);
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
            for (int pg = 0; pg < P; ++pg) {
                unit[pg] = 15;                 // s from 2^-7 to 2, as values of a usual spread have
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    z[n][0] = z[n][1] = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[pg][i][n][0] = o[pg][i][n][1] = o[pg][i][n][2] = o[pg][i][n][3] = 0.0f;
                }
            }
            clear = min(clear, __shfl_xor_sync(~0u, clear, 1));
            clear = min(clear, __shfl_xor_sync(~0u, clear, 2));
            __syncthreads();               // the other warps' rows of the queries
            prepare_queries(queries + cq * q_bytes);
            cq = cq + 1 == kQueries ? 0 : cq + 1;
            __syncthreads();
            if (NB == 1) {
#pragma unroll
                for (int pg = 0; pg < (NB == 1 ? P : 0); ++pg) {
                    held[pg][0] = frag[(pg * 2) * 32 + lane];
                    held[pg][1] = frag[(pg * 2 + 1) * 32 + lane];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    held_fac[e] = facs[2 * (lane & 3) + e];
#pragma unroll
                    for (int pg = 0; pg < (NB == 1 ? P : 0); ++pg) held_sum[pg][e] = qsum[(2 * (lane & 3) + e) * P + pg];
                }
            }
        }
        __syncwarp();
        const int key0 = p.step * kStep + warp * KW;
        uint8_t *st = ring + stage * kStageBytes;
        if (key0 < nkeys) {
            const uint32_t st_at = ring_at + stage * kStageBytes;
            if (key0 + KW > clear) stage_products(std::true_type{}, st, st_at, key0);
            else stage_products(std::false_type{}, st, st_at, key0);
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
            for (int n = 0; n < NB; ++n) {     // 8 rows at a time
                if (n > 0 && tiles <= n) break;
                float *mine = reinterpret_cast<float *>(st);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 2 * (lane & 3) + e;
                    float sum = l[n][e];
                    sum += __shfl_xor_sync(~0u, sum, 4);
                    sum += __shfl_xor_sync(~0u, sum, 8);
                    sum += __shfl_xor_sync(~0u, sum, 16);
                    if (lane < 4) {
                        const bool none = (blind >> (2 * n + e)) & 1;
                        stats[(warp * RT + n * 8 + r) * 2] = none ? -INFINITY : m[n][e];
                        stats[(warp * RT + n * 8 + r) * 2 + 1] = none ? 0.0f : sum;
                    }
#pragma unroll
                    for (int pg = 0; pg < P; ++pg) {
                        const float zs = __shfl_sync(~0u, z[n][e], 4 * pg + (lane & 3));
                        // codes' units: 2^24 and 2^20, over inv = 2^(14 - unit)
                        const float f0 = power2(10 + unit[pg]), f1 = power2(6 + unit[pg]);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int at = pg * 64 + half * 32 + 4 * (lane >> 2);
                            *reinterpret_cast<float4 *>(mine + r * D + (at ^ ((lane & 3) << 3))) =
                                make_float4(fmaf(o[pg][0][n][2 * half + e], f0, zs), fmaf(o[pg][1][n][2 * half + e], f1, zs),
                                            fmaf(o[pg][2][n][2 * half + e], f0, zs), fmaf(o[pg][3][n][2 * half + e], f1, zs));
                        }
                    }
                }
                __syncthreads();
                constexpr int LR = D / 4, RW = 32 / LR;   // lanes of a row, rows of a warp pass
                const float *all = reinterpret_cast<const float *>(smem + stage * kStageBytes);
                for (int r = warp * RW + lane / LR; r < 8; r += kWarps * RW) {
                    const int row = p.tile * RT + n * 8 + r;
                    if (row >= rows) break;
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stats[(w * RT + n * 8 + r) * 2]);
                    const float base = base_of(top);
                    const int c = (lane % LR) * 4, cs = c ^ (((r >> 1) & 3) << 3);
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    float sum = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float2 ml = *reinterpret_cast<const float2 *>(stats + (w * RT + n * 8 + r) * 2);
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
                        const int t = token_of(A, row), gq = row - t * G;
                        const int64_t at = (int64_t(p.b) * J.batch.T + t) * J.q_heads + int64_t(p.h) * G + gq;
                        const float inv = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
                        store_out<T>(J, at * D + c, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                        if (J.lse && lane % LR == 0) J.lse[at] = lse_of(top, sum);
                    } else {
                        *reinterpret_cast<float4 *>(part + (n * 8 + r) * D + c) = v;
                        if (lane % LR == 0)
                            *reinterpret_cast<float2 *>(part + RT * D + (n * 8 + r) * 2) = make_float2(top, sum);
                    }
                }
                __syncthreads();
            }
            if (!direct && J.batch.prefix_len == 0) {
                // (the warp's other stages are free where nothing is left to load)
                const bool all = u + 1 == hi;
                join_apart<T, D, RT>(A, S, p, rows, W, count, scratch, all ? ring : st,
                                     (all ? kStages : 1) * kStageBytes / 512);
            }
            fresh = true;
        }
        load_next(stage);
        if (++stage == kStages) stage = 0;
        ++p.step;
        ++u;
    }
    // the join waits for this grid alone and reads the prefix kernel's results too: one CTA
    // ends after that kernel
    if (A.tc_items && blockIdx.x == 0) pdl_wait();
    tc::cp_async_wait<0>();
}

// Dynamic shared memory of a CTA: rings, query tiles, their operands and row data, warps'
// (m, l), the batch.
size_t smem_of(const Args &A) {
    const int D = A.J.cache.head_dim, P = D / kGroup, stage = KW * (D + 8 * P);
    return size_t(kWarps) * kStages * stage + size_t(kStages + 1) * A.RT * D * 2 + size_t(A.RT / 8) * P * 1024 +
           A.RT * 4 * (1 + P) + kWarps * A.RT * 8 + kWarps * 4 + (size_t(A.J.batch.B) * 3 + 1) * 4;
}

// A prefix that many rows read goes through the tensor cores' kernel, which wants 16 bits: written out once a
// call, each value as two fp16 (s c + z to 22 bits), and the queries beside it as fp16 in units of
// their own.  Weights are rounded once there, to fp16.
constexpr int kPage = 128;         // keys of a page of that copy
// Measured, here and on tiles of 16 rows (us in all, own keys of 50 to 200): 5 heads of 128, 300 rows, prefix
// of 1000 and 16000: 29 and 78, 36 and 161; 128 rows, 1000 and 4000: 24 and 30, 23 and 36; 8 heads of 64, 300 rows, 300
// and 4000: 22 and 34, 22 and 48; 126 rows, 4000: 29, 26; one head of 128, 296 rows, 1000 and 4000: 19 and 21, 17
// and 27.  (A tile of 128 rows is filled in pairs; the copy is held to 1 GB.)
bool prefix_written_out(const trit_attn_job &J) {
    const int64_t rows = int64_t(J.batch.B) * J.batch.T * (J.q_heads / J.cache.heads);
    const int64_t columns = J.batch.prefix_len * J.cache.heads * J.cache.head_dim;
    return rows > 96 && columns <= int64_t(1) << 27 && double(rows) * double(columns) >= (rows > 128 ? 1e8 : 3.2e8);
}

Args layout(const trit_attn_job &J) { return layout_of(J, kStep, smem_of, prefix_written_out(J), 16, true); }

// What the copy takes of the workspace, behind the partial results: K, V, the queries, their units, pages' numbers.
struct Copy {
    int64_t pages, vectors, k, v, q, units, table, end;      // offsets in bytes
};
Copy copy_of(const Args &A) {
    const trit_attn_job &J = A.J;
    Copy c = {};
    c.k = head_bytes(A) + part_bytes(A) + (A.tc_items ? prefix_part_bytes(A) : 0);
    c.end = c.k;
    if (!A.tc_items) return c;
    c.k = (c.k + 255) / 256 * 256;
    c.pages = (J.batch.prefix_len + kPage - 1) / kPage;
    c.vectors = c.pages * kPage * J.cache.heads;
    c.v = c.k + c.vectors * J.cache.head_dim * 4;
    c.q = c.v + c.vectors * J.cache.head_dim * 4;
    const int64_t rows = int64_t(J.batch.B) * J.batch.T * J.q_heads;
    c.units = c.q + rows * J.cache.head_dim * 2;
    c.table = c.units + rows * 4;
    c.end = (c.table + c.pages * 4 + 255) / 256 * 256;
    return c;
}

struct WriteArgs {
    trit_attn_job J;                 // its cache: the codes, strides in vectors
    const uint8_t *k_scale, *v_scale;
    uint32_t *err;
    __half *k, *v, *q;               // [heads][pages * kPage][2 D] (hi, lo), [B T][Hq][D]
    float *units;
    int32_t *table;
    uint32_t flip, keep;             // the sign of scale, and 0 where it is 0, on pairs of q
    int32_t keys;                    // pages * kPage
    int32_t q_blocks;                // blocks of the queries, the first ones
    int32_t page_shift;
};

// What is finite in fp16's range, the rest as it is.
__device__ __forceinline__ float held(float x) { return fabsf(x) < INFINITY ? fminf(fmaxf(x, -65504.0f), 65504.0f) : x; }

// Eight columns a lane, vectors of K and then of V, each by head and key.  Bound by latency and by its stores: 4
// bytes a code.
constexpr int kWriteThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kWriteThreads) write_out_kernel(const __grid_constant__ WriteArgs A) {
    const trit_attn_job &J = A.J;
    constexpr int L = D / 8;
    pdl_wait();
    pdl_launch();
    if (int(blockIdx.x) < A.q_blocks) {       // a lane D / 32 columns of a row
        const int lane = threadIdx.x & 31;
        const int64_t row = int64_t(blockIdx.x) * (kWriteThreads / 32) + (threadIdx.x >> 5);
        if (row >= int64_t(J.batch.B) * J.batch.T * J.q_heads) return;
        const int64_t token = row / J.q_heads;
        constexpr int C = D / 64;             // pairs of columns
        const uint32_t *src = reinterpret_cast<const uint32_t *>(static_cast<const T *>(J.q) + token * J.q_stride + (row - token * J.q_heads) * D) + lane * C;
        float2 x[C];
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            x[i] = unpack16<T>((__ldg(src + i) & A.keep) ^ A.flip);
            most = fmaxf(most, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
        // the largest column to [2^14, 2^15)
        int e = 14 - ((__float_as_int(most) >> 23) - 127);
        e = e > 100 ? 100 : e < -100 ? -100 : e;
        const float f = power2(e);
        uint32_t *dst = reinterpret_cast<uint32_t *>(A.q + row * D) + lane * C;
#pragma unroll
        for (int i = 0; i < C; ++i) dst[i] = pack16<__half>(x[i].x * f, x[i].y * f);
        if (lane == 0) A.units[row] = power2(-e);
        return;
    }
    const int block = int(blockIdx.x) - A.q_blocks;
    if (block == 0)
        for (int i = threadIdx.x; i < A.keys / kPage; i += kWriteThreads) A.table[i] = i;
    const int64_t at = (int64_t(block) * kWriteThreads + threadIdx.x) / L, half = int64_t(A.keys) * J.cache.heads;
    if (at >= 2 * half) return;
    const bool is_v = at >= half;
    const int64_t vec = is_v ? at - half : at;
    const int h = int(vec / A.keys), key = int(vec - int64_t(h) * A.keys), sub = threadIdx.x % L;
    uint32_t word = 0;
    __half2 sz = {};
    if (key < J.batch.prefix_len) {
        const int col = A.page_shift >= 0 ? key >> A.page_shift : key / J.cache.page_size;
        const int page = __ldg(J.batch.prefix_table + col);
        if (page >= 0 && page < J.cache.pages) {
            const int64_t from = page * J.cache.page_stride + int64_t(key - col * J.cache.page_size) * J.cache.slot_stride + h * J.cache.head_stride;
            word = __ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(is_v ? J.cache.v : J.cache.k) + from * (D / 2)) + sub);
            sz = __ldg(reinterpret_cast<const __half2 *>((is_v ? A.v_scale : A.k_scale) + from * (D / 16)) + sub / 8);
        } else if (sub == 0) {
            raise_flag(A.err, TRIT_ERR_INDEX);
        }
    }
    const float2 f = __half22float2(sz);
    const float s[4] = {f.x, f.x * 0.0625f, f.x * 0.00390625f, f.x * 0.000244140625f};
    uint32_t w[4], rest[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            // 2^23 + c 16^n, exactly, by its bits; what is finite stays so
            const int n = 2 * i + j;
            const float c = __uint_as_float(0x4b000000u | ((n < 4 ? word : word >> 16) & (15u << (4 * (n & 3))))) - 8388608.0f;
            y[j] = fmaf(c, s[n & 3], f.y);
        }
        const float2 most = {held(y[0]), held(y[1])};
        w[i] = pack16<__half>(most.x, most.y);
        const float2 hi = unpack16<__half>(w[i]);
        rest[i] = pack16<__half>(fabsf(y[0]) < INFINITY ? held(y[0] - hi.x) : 0.0f, fabsf(y[1]) < INFINITY ? held(y[1] - hi.y) : 0.0f);
    }
    __half *const to = (is_v ? A.v : A.k) + vec * 2 * D + sub * 8;
    *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(to + D) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
}

// The copy, and the tensor cores' kernel over it.
template <typename T, int D>
cudaError_t launch_written(const Args4 &A4, cudaStream_t s) {
    Args A = A4.A;
    const Copy c = copy_of(A);
    uint8_t *ws = reinterpret_cast<uint8_t *>(A.count);
    WriteArgs W = {};
    W.J = A.J;
    W.k_scale = A4.k_scale;
    W.v_scale = A4.v_scale;
    W.err = A.err;
    W.k = reinterpret_cast<__half *>(ws + c.k);
    W.v = reinterpret_cast<__half *>(ws + c.v);
    W.q = reinterpret_cast<__half *>(ws + c.q);
    W.units = reinterpret_cast<float *>(ws + c.units);
    W.table = reinterpret_cast<int32_t *>(ws + c.table);
    W.flip = A.J.scale < 0.0f ? 0x80008000u : 0u;
    W.keep = A.J.scale == 0.0f ? 0u : 0xffffffffu;
    W.keys = int32_t(c.pages * kPage);
    W.page_shift = A.page_shift;
    const int64_t rows = int64_t(A.J.batch.B) * A.J.batch.T * A.J.q_heads;
    W.q_blocks = int32_t((rows + kWriteThreads / 32 - 1) / (kWriteThreads / 32));
    const int64_t lanes = 2 * c.vectors * (D / 8);
    const cudaError_t e = launch_pdl(write_out_kernel<T, D>, dim3(unsigned(W.q_blocks + (lanes + kWriteThreads - 1) / kWriteThreads)),
                                     dim3(kWriteThreads), 0, s, W);
    if (e != cudaSuccess) return e;
    A.scale2 = A.J.scale == 0.0f ? 1.0f : fabsf(A4.scale2);
    A.flip = 0;
    A.keep = 0xffffffffu;
    A.q_units = W.units;
    A.J.q = W.q;
    A.J.q_stride = int64_t(A.J.q_heads) * D;
    A.J.cache.k = W.k;
    A.J.cache.v = W.v;
    A.J.cache.slot_stride = D;
    A.J.cache.page_stride = kPage * D;
    A.J.cache.head_stride = int64_t(W.keys) * D;
    A.J.cache.pages = int32_t(c.pages);
    A.J.cache.page_size = kPage;
    A.J.cache.dtype = TRIT_F16;
    A.J.batch.prefix_table = W.table;
    return launch_prefix(A, s);
}

// The job as the shared layout knows it: a cache of codes, strides in vectors.
trit_attn_job plain_of(const trit_attn4_job &J) {
    trit_attn_job p = {};
    p.cache.k = J.cache.k;
    p.cache.v = J.cache.v;
    p.cache.page_stride = J.cache.page_stride;
    p.cache.head_stride = J.cache.head_stride;
    p.cache.slot_stride = J.cache.slot_stride;
    p.cache.pages = J.cache.pages;
    p.cache.heads = J.cache.heads;
    p.cache.page_size = J.cache.page_size;
    p.cache.head_dim = J.cache.head_dim;
    p.cache.dtype = J.dtype;
    p.batch = J.batch;
    p.q = J.q;
    p.out = J.out;
    p.lse = J.lse;
    p.q_stride = J.q_stride;
    p.scale = J.scale;
    p.q_heads = J.q_heads;
    p.out_dtype = J.out_dtype;
    return p;
}

template <typename T, int D, int NB>
cudaError_t launch(const Args4 &A4, cudaStream_t s) {
    const Args &A = A4.A;
    const auto kernel = attn4_kernel<T, D, NB>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 180 * 1024);
    // (the own keys' kernel depends on nothing of the prefix's and may run beside it)
    if (e == cudaSuccess && A.tc_items) e = launch_written<T, D>(A4, s);
    if (e == cudaSuccess) e = launch_pdl(kernel, dim3(unsigned(A.grid)), dim3(kThreads), smem_of(A), s, A4);
    if (e != cudaSuccess || A.J.batch.prefix_len == 0) return e;
    const int64_t joins = int64_t(A.J.batch.B) * A.J.cache.heads * ((A.R + 3) / 4);
    if (joins <= 2 * kSms) return launch_pdl(join_kernel<T, D, 4>, dim3(unsigned(joins)), dim3(4 * D), 0, s, A);
    return launch_pdl(join_kernel<T, D, 1>, dim3(unsigned(joins)), dim3(D), 0, s, A);
}

template <typename T>
cudaError_t launch_t(const Args4 &A4, cudaStream_t s) {
    const int RT = A4.A.RT;
    if (A4.A.J.cache.head_dim == 128)
        return RT == 8 ? launch<T, 128, 1>(A4, s) : launch<T, 128, 2>(A4, s);
    return RT == 8 ? launch<T, 64, 1>(A4, s) : launch<T, 64, 2>(A4, s);
}

}  // namespace
}  // namespace attn

int64_t attn4_workspace_bytes(const trit_attn4_job &J) {
    return attn::copy_of(attn::layout(attn::plain_of(J))).end;
}

cudaError_t launch_attn_paged4(const trit_attn4_job &J, uint32_t *err, cudaStream_t s) {
    attn::Args4 A4;
    attn::Args &A = A4.A;
    A = attn::layout(attn::plain_of(J));
    A.err = err;
    A4.k_scale = static_cast<const uint8_t *>(J.cache.k_scale);
    A4.v_scale = static_cast<const uint8_t *>(J.cache.v_scale);
    A4.scale2 = J.scale * 1.4426950408889634f;
    A4.runs = J.cache.slot_stride == 1 && A.page_shift >= 5;
    uint8_t *ws = static_cast<uint8_t *>(J.workspace);
    A.count = reinterpret_cast<uint32_t *>(ws);
    A.cum = reinterpret_cast<int32_t *>(ws + attn::kCountBytes);
    A.parts = reinterpret_cast<float *>(ws + attn::head_bytes(A));
    A.tc_parts = A.parts + attn::part_bytes(A) / 4;
    return J.dtype == TRIT_BF16 ? attn::launch_t<__nv_bfloat16>(A4, s) : attn::launch_t<__half>(A4, s);
}

}  // namespace trit
