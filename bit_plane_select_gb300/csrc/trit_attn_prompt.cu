// trit_attn_prompt: causal attention of packed prompts on the 5th-generation tensor
// cores.
//
// With 4 D Hq flops a pair of query and key on 2 D (2 Hq + 2 Hkv) bytes a token, prompts
// of more than a few hundred tokens are bound by the tensor pipe, and beside it by the
// exponentials.  A tile is 128 rows, a softmax of one row per thread (no shuffles): S (128 x 128
// fp32 in tensor memory) is overwritten in place by P (16-bit, the operand of the second
// product), O accumulates beside it and is rescaled only when a row's maximum grew by more
// than 2^8 since its base was fixed.  These steps wait for one another, so an SM runs two of them
// at a time, one's products under the other's softmax: two CTAs, a tile each, which
// also covers the beginning and end of a tile by the other's work; or, where there are
// fewer tiles than SMs, one CTA whose two streams take a tile's blocks of keys by turns
// (TURNS) and are joined at the end.  (Measured, us: one prompt of 16384 tokens, 20 query heads over 5 of
// 128: 849 in short bursts, 910 call after call under the power limit; in bursts two tiles of one CTA sharing the loads of K and V 965.  700 tokens: 12.4 by turns, 13.9 a
// tile per CTA.)  P goes to the products in halves of 64 keys (in quarters 855 to 890 us, whole 928):
// every store to tensor memory is waited for, and takes its turn behind the products under way.
//
// A row is a token and one of the G query heads that share a key head: 128 / G tokens'
// rows fill a tile, so one K and V tile serves them all, a prompt's diagonal cuts off little
// (a tile of G = 4 covers 32 tokens), and short prompts leave few rows empty.  Q, K and V
// come by TMA; the box (64 columns, G heads, 128 / G tokens) lays Q out in that order.
//
// Keys come in blocks of 128 in rising order.  Only the last blocks, past the first row's
// limit, are masked.  There a value that some row must not see may be infinite or NaN, and its
// P = 0 would not keep it away (0 * inf is NaN): the warp that loads V looks such
// blocks through on their way, puts 0 in the place of what is not finite, and leaves a note
// on which the rows add up what they do see, one by one, at the end.
#include "trit_attn.cuh"
#include "trit_attn_tc.cuh"

namespace trit {
namespace attn {
namespace {

constexpr int kRows = 128;
constexpr float kGrow = 8.0f;      // log2 of the growth of a maximum that O tolerates

template <int D>
__host__ __device__ constexpr int tile_bytes() { return kBlockKeys * D * 2; }

template <int D, bool TURNS>
struct Shape {
    static constexpr int kStreams = TURNS ? 2 : 1;
    // tiles of K and V in flight: with D = 128 and two CTAs one of each
    static constexpr int kRing = !TURNS && D == 128 ? 2 : 4;
    static constexpr int kMmaWarp = 4 * kStreams;         // and the next: an issuing warp per stream
    static constexpr int kLoadWarp = kMmaWarp + 2;        // and the next: Q's and K's copies, and V's
    static constexpr int kThreads = 128 * kStreams + 128;
    // Registers: the softmax warpgroups, which hold a row of S, take some of the last one's:
    // 256 * 216 + 128 * 72 = 384 * 168, 128 * 200 + 128 * 56 = 256 * 128.
    static constexpr int kLaunchRegs = kStreams == 2 ? 168 : 128;
    static constexpr int kTmemCols = 256 * kStreams;      // S of the streams, 128 columns each, and O
    static constexpr size_t kSmem = 1024 + size_t(1 + kRing) * tile_bytes<D>() + 256 + (TURNS ? kRows * 8 : 0);
};
template <int STREAMS>
__device__ __forceinline__ void more_registers() {
    if (STREAMS == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
}
template <int STREAMS>
__device__ __forceinline__ void fewer_registers() {
    if (STREAMS == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
}

struct PromptArgs {
    trit_prompt_job J;
    uint32_t *err;
    float scale2;            // scale log2(e)
    int32_t G;               // query heads per key head
    int32_t heads;           // of a tile: min(G, 128)
    int32_t parts;           // tiles that the G heads of a key head take
    int32_t page;            // parts * key heads: items of the same tokens
    int32_t unit;            // tokens of a tile: 128 / heads
    int32_t sorted;          // whether the items come by falling length
};

// Sequence b's queries and keys; none where the starts are not in order.
struct Span {
    int32_t q0, nq, k0, nk;
};
__device__ __forceinline__ Span span_of(const PromptArgs &A, int b, bool *bad) {
    const trit_prompt_job &J = A.J;
    const int32_t *ks = J.k_starts ? J.k_starts : J.q_starts;
    Span s{J.q_starts[b], J.q_starts[b + 1], ks[b], ks[b + 1]};
    const bool ok = s.q0 >= 0 && s.nq >= s.q0 && s.nq <= J.q_rows && s.k0 >= 0 && s.nk >= s.k0 && s.nk <= J.k_rows;
    s.nq = ok ? s.nq - s.q0 : 0;
    s.nk = ok ? s.nk - s.k0 : 0;
    *bad = !ok;
    return s;
}

// The k-th tile's tokens (a unit) of the batch, found by a whole warp: its sequence's span, and which
// of the sequence's it is (-1: there are fewer).
__device__ __forceinline__ int lane_scan(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += x;
    }
    return v;
}
__device__ __forceinline__ Span from_lane(const Span &s, int who) {
    return Span{__shfl_sync(~0u, s.q0, who), __shfl_sync(~0u, s.nq, who), __shfl_sync(~0u, s.k0, who),
                __shfl_sync(~0u, s.nk, who)};
}
// Of 32 sequences, one a lane, in their order: where starts fall, some may have rows in common and more tiles than the
// grid.  One that has rows of a sequence before it is left out too; `taken` ends the rows of those that are not.
__device__ __forceinline__ void keep_apart(Span &s, int lane, int32_t &taken) {
    for (int i = 0; i < 32; ++i) {
        const int32_t q0 = __shfl_sync(~0u, s.q0, i), n = __shfl_sync(~0u, s.nq, i);
        if (n == 0) continue;
        if (q0 >= taken) taken = q0 + n;
        else if (lane == i) s.nq = 0;
    }
}
// In the order of the sequences, 32 at a time, a sequence's last units first.
__device__ __forceinline__ int find_in_order(const PromptArgs &A, int k, int lane, bool report, Span &me) {
    int unit = -1;
    int32_t taken = -1;                           // (-1: all starts so far are in order)
    for (int b0 = 0; b0 < A.J.B; b0 += 32) {
        bool bad = false;
        Span s{0, 0, 0, 0};
        if (b0 + lane < A.J.B) s = span_of(A, b0 + lane, &bad);
        if (bad && report) raise_flag(A.err, TRIT_ERR_INDEX);
        if (taken >= 0 || __any_sync(~0u, bad)) {
            if (taken < 0) taken = b0 ? A.J.q_starts[b0] : 0;
            keep_apart(s, lane, taken);
        }
        const int n = (s.nq + A.unit - 1) / A.unit, inc = lane_scan(n, lane), all = __shfl_sync(~0u, inc, 31);
        if (unit < 0 && k < all) {
            const int who = __ffs(int(__ballot_sync(~0u, k < inc))) - 1;
            me = from_lane(s, who);
            unit = __shfl_sync(~0u, inc, who) - 1 - k;
            if (!report) break;                   // (the CTA that reports looks at all starts)
        }
        k -= all;
    }
    return unit;
}
// Of up to 32 sequences by falling number of key blocks, so that the longest start first: a
// division per sequence tells how many units have at least x blocks, and a bisection
// over x finds the k-th.
__device__ __forceinline__ int find_by_length(const PromptArgs &A, int k, int lane, bool report, Span &me) {
    bool bad = false;
    Span s{0, 0, 0, 0};
    if (lane < A.J.B) s = span_of(A, lane, &bad);
    if (bad && report) raise_flag(A.err, TRIT_ERR_INDEX);
    if (__any_sync(~0u, bad)) {
        int32_t taken = 0;
        keep_apart(s, lane, taken);
    }
    const int units = (s.nq + A.unit - 1) / A.unit;
    // the lane's first unit with at least x blocks (those behind it have them too); units whose last token sees no
    // key have none
    auto first_with = [&](int x) {
        if (x <= 0) return 0;
        const int need = (x - 1) * kBlockKeys + 1 - (s.nk - s.nq);      // tokens up to its last
        if (need > s.nq) return units;
        return need <= A.unit ? 0 : (need + A.unit - 1) / A.unit - 1;
    };
    auto with = [&](int x) { return int(__reduce_add_sync(~0u, unsigned(units - first_with(x)))); };
    if (k >= with(0)) return -1;
    int lo = 0, hi = int(__reduce_max_sync(~0u, unsigned(s.nq > 0 ? (s.nk + kBlockKeys - 1) / kBlockKeys : 0)));
    while (lo < hi) {                             // with(lo) > k >= with(hi + 1)
        const int mid = (lo + hi + 1) >> 1;
        if (with(mid) > k) lo = mid;
        else hi = mid - 1;
    }
    k -= with(lo + 1);                            // among those with just lo blocks
    const int from = first_with(lo), n = first_with(lo + 1) - from, inc = lane_scan(n, lane);
    const int who = __ffs(int(__ballot_sync(~0u, k < inc))) - 1;
    me = from_lane(s, who);
    return __shfl_sync(~0u, from + k - (inc - n), who);
}

__device__ __forceinline__ void tma_rows(void *dst, const CUtensorMap *map, int x, int head, int row, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2,%3,%4}], [%5];" ::
            "r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(head), "r"(row), "r"(smem_u32(bar))
        : "memory");
}
// The address of the tensor memory is in shared memory: a barrier of the softmax and
// issuing warps.
template <int STREAMS>
__device__ __forceinline__ void tmem_ready() { asm volatile("bar.sync 1, %0;" ::"n"(160 * STREAMS) : "memory"); }

template <typename T>
__host__ __device__ constexpr uint32_t inf_bits() { return 0x7c00u; }
template <>
__host__ __device__ constexpr uint32_t inf_bits<__nv_bfloat16>() { return 0x7f80u; }
// Two 16-bit values, those that are infinite or NaN replaced by 0.
template <typename T>
__device__ __forceinline__ uint32_t finite_pair(uint32_t v) {
    constexpr uint32_t kInf = inf_bits<T>();
    return ((v & 0x7fffu) >= kInf ? 0u : v & 0xffffu) | (((v >> 16) & 0x7fffu) >= kInf ? 0u : v & 0xffff0000u);
}

// 0 v + sum in 16 bits: 0, or NaN once a value was infinite or NaN.
template <typename T>
__device__ __forceinline__ uint32_t times0(uint32_t v, uint32_t sum) {
    uint32_t d;
    if (sizeof(T) && type_bits<T>()) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(0u), "r"(sum));
    else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(0u), "r"(sum));
    return d;
}

template <typename T, int D, bool TURNS>
__global__ void __launch_bounds__(Shape<D, TURNS>::kThreads, TURNS ? 1 : 2)
    prompt_kernel(const __grid_constant__ PromptArgs A, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using Sh = Shape<D, TURNS>;
    constexpr int kTile = tile_bytes<D>(), kRing = Sh::kRing, kMmaWarp = Sh::kMmaWarp, kLoadWarp = Sh::kLoadWarp;
    constexpr int kTmemO = 128 * Sh::kStreams;            // S of stream s at 128 s, O at 128 s of the second half
    uint8_t *qs = smem, *ring = smem + kTile;
    uint64_t *full = reinterpret_cast<uint64_t *>(ring + kRing * kTile);
    uint64_t *empty = full + kRing;
    uint64_t *s_full = empty + kRing;    // stream's S is in tensor memory
    uint64_t *p_full = s_full + 2;       // [stream][half]: P of 64 keys each is
    uint64_t *o_full = p_full + 4;       // stream's O is finished
    uint64_t *pv_done = o_full + 2;      // stream's product into O has completed
    uint64_t *q_full = pv_done + 2;
    uint64_t *tail = q_full + 1;         // the copies of a V block that is looked through
    constexpr int kBars = 2 * kRing + 12;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tail + 1);
    uint32_t *timed_out = tmem_slot + 1;
    uint32_t *odd = tmem_slot + 2;       // V held an infinity or NaN in a block that is masked

    const trit_prompt_job &J = A.J;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kMmaWarp && lane < kBars) {       // a barrier per lane, in the order above
        const int i = lane;
        const bool by_warps = i >= 2 * kRing + 2 && i < 2 * kRing + 6;       // p_full
        mbar_init(full + i, by_warps ? 4u : 1u);
        if (i == 0) *timed_out = *odd = 0;
        fence_barrier_init();
    }
    if (warp == kLoadWarp && lane < 3)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap) : "memory");
    __syncthreads();
    if (warp == kMmaWarp) {       // beside the search for the item
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(Sh::kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    auto free_tmem = [&]() {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tmem_slot), "r"(Sh::kTmemCols));
    };
    pdl_wait();
    pdl_launch();

    // the item: a tile of one sequence and a key head
    const int unit_at = int(blockIdx.x) / A.page;
    const int item = int(blockIdx.x) - unit_at * A.page, h = item / A.parts, part = item - h * A.parts;
    Span me{0, 0, 0, 0};
    const bool report = blockIdx.x == 0 && warp == 0;
    const int which = A.sorted ? find_by_length(A, unit_at, lane, report, me) : find_in_order(A, unit_at, lane, report, me);
    if (which < 0) {                              // more CTAs than units: the same for every warp
        if (warp == kMmaWarp) free_tmem();
        return;
    }
    const int t0 = which * A.unit;                // the item's first token
    const int behind = me.nk - me.nq;             // query t sees keys 0 .. t + behind
    // blocks of the CTA, up to its last token's limit, and of the streams
    const int last = min(t0 + A.unit, me.nq) + behind, n = last > 0 ? (last + kBlockKeys - 1) / kBlockKeys : 0;
    const int n0 = TURNS ? (n + 1) / 2 : n, n1 = TURNS ? n / 2 : 0;
    const int first_limit = max(0, behind + t0 + 1);
    const int partial = first_limit / kBlockKeys;              // blocks from here on are hidden from some row

    if (warp >= kLoadWarp) {
        fewer_registers<Sh::kStreams>();
        const bool is_v = warp > kLoadWarp;
        if (!is_v && lane == 0 && n > 0) {
            const uint32_t bytes = uint32_t(A.heads * A.unit * 128);
            mbar_arrive_expect_tx(q_full, (D / 64) * bytes);
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
                tma_rows(qs + i * (kRows * 128), &qmap, i * 64, h * A.G + part * 128, me.q0 + t0, q_full);
        }
        __syncwarp();
        const CUtensorMap *map = is_v ? &vmap : &kmap;
        for (int j = 0; j < n; ++j) {
            const int at = 2 * j + is_v, s = at % kRing;
            const bool look = is_v && j >= partial;
            uint64_t *bar = look ? tail : &full[s];
            uint8_t *st = ring + s * kTile;
            if (!warp_wait(&empty[s], ((at / kRing) & 1) ^ 1, timed_out)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, kTile);
#pragma unroll
                for (int half = 0; half < D / 64; ++half)
                    tma_rows(st + half * (kBlockKeys * 128), map, half * 64, h, me.k0 + j * kBlockKeys, bar);
            }
            __syncwarp();
            if (look) {
                if (!warp_wait(tail, (j - partial) & 1, timed_out)) break;
                // from the first key that some row must not see: 0 v + 0 + .. is 0 where all are finite
                uint4 *v = reinterpret_cast<uint4 *>(st);
                const int from = max(0, first_limit - j * kBlockKeys);
                uint32_t sum[4] = {0, 0, 0, 0};
                for (int half = 0; half < D / 64; ++half)
#pragma unroll 4
                    for (int i = half * (kBlockKeys * 8) + from * 8 + lane; i < (half + 1) * (kBlockKeys * 8); i += 32) {
                        const uint4 w = v[i];
                        sum[0] = times0<T>(w.x, sum[0]);
                        sum[1] = times0<T>(w.y, sum[1]);
                        sum[2] = times0<T>(w.z, sum[2]);
                        sum[3] = times0<T>(w.w, sum[3]);
                    }
                if (__any_sync(~0u, ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu) != 0)) {
                    for (int i = lane; i < kTile / 16; i += 32) {
                        uint4 w = v[i];
                        w.x = finite_pair<T>(w.x); w.y = finite_pair<T>(w.y);
                        w.z = finite_pair<T>(w.z); w.w = finite_pair<T>(w.w);
                        v[i] = w;
                    }
                    *reinterpret_cast<volatile uint32_t *>(odd) = 1;
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
            }
        }
    } else if (warp >= kMmaWarp + Sh::kStreams) {
        fewer_registers<Sh::kStreams>();        // (one stream: nothing for the second issuing warp)
    } else if (warp >= kMmaWarp) {
        fewer_registers<Sh::kStreams>();
        tmem_ready<Sh::kStreams>();
        tc_fence_after();
        const uint32_t tmem = *tmem_slot;
        // stream s: S of its first block, then per block O += P V and S of the next,
        // which takes the place of P once that product has completed.  The whole warp
        // walks the loop (uniform values, so the operands are in uniform registers
        // when a product is issued); one elected lane issues.
        const int s = TURNS ? warp - kMmaWarp : 0, mine = s ? n1 : n0;      // (one stream: known when compiled)
        const bool leader = elect_one();
        const uint32_t qlo = desc_lo(smem_u32(qs)) | kDescK;
        const uint32_t rk = desc_lo(smem_u32(ring)) | kDescK, rv = desc_lo(smem_u32(ring)) | kDescMn;
        const uint32_t sp = tmem + s * 128, o = tmem + kTmemO + s * 128;
        auto tile_there = [&](int at) -> bool { return warp_wait(&full[at % kRing], (at / kRing) & 1, timed_out); };
        // (K of the stream's block i is the ring's tile k_at(i), V the next: with two streams each stage of
        // the ring serves one of them, so that none misses a phase of its barriers)
        auto k_at = [&](int i) { return 2 * (Sh::kStreams * i + s); };
        auto issue_s = [&](int i) {
            const int st = k_at(i) % kRing;
            tc_fence_after();
            const uint32_t b = rk + st * (kTile >> 4);
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk / 4) * (kBlockKeys * 128 >> 4) + (kk % 4) * 2;
                    mma_ss(sp, qlo + off, b + off, idesc_s<T>(), kk > 0);
                }
                mma_commit(&s_full[s]);
                mma_commit(&empty[st]);
            }
            __syncwarp();
        };
        bool ok = n == 0 || warp_wait(q_full, 0, timed_out);
        if (ok && mine > 0) {
            ok = tile_there(k_at(0));
            if (ok) issue_s(0);
        }
        for (int i = 0; ok && i < mine; ++i) {
            const int at = k_at(i) + 1, st = at % kRing;
            ok = tile_there(at);
            const uint32_t b = rv + st * (kTile >> 4);
#pragma unroll
            for (int part2 = 0; part2 < 2; ++part2) {
                ok = ok && warp_wait(&p_full[2 * s + part2], i & 1, timed_out);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 4 * part2; kk < 4 * part2 + 4; ++kk)
                        mma_ts(o, sp + kk * 8, b + kk * (2048 >> 4), idesc_o<T, D>(), i > 0 || kk > 0);
                }
                __syncwarp();
            }
            if (!ok) break;
            const bool last = i + 1 == mine;
            if (leader) {
                mma_commit(last ? &o_full[s] : &pv_done[s]);
                mma_commit(&empty[st]);
            }
            __syncwarp();
            if (!last) {
                ok = tile_there(k_at(i + 1)) && warp_wait(&pv_done[s], i & 1, timed_out);
                if (ok) issue_s(i + 1);
            }
        }
    } else {
        // softmax: stream s, row r of its tile (tensor-memory lane r)
        more_registers<Sh::kStreams>();
        const int s = TURNS ? warp >> 2 : 0, r = threadIdx.x & 127;
        const uint32_t quarter = uint32_t((warp & 3) * 32) << 16;
        tmem_ready<Sh::kStreams>();
        tc_fence_after();
        const uint32_t tmem = *tmem_slot;
        const float scale2 = A.scale2;
        const int mine = s ? n1 : n0;                  // this stream's blocks
        const int tile_t = r / A.heads, g = part * 128 + r - tile_t * A.heads, t = t0 + tile_t;
        const bool there = tile_t < A.unit && t < me.nq && g < A.G;
        const int limit = there ? max(0, t + behind + 1) : 0;       // keys that the row sees
        float m = -INFINITY, m_raw = 0.0f, l = 0.0f;      // m: m_raw scaled
        bool ok = true;
        for (int i = 0; i < mine; ++i) {
            ok = warp_wait(&s_full[s], i & 1, timed_out);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sa = tmem + s * 128 + quarter;
            uint32_t v[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(sa + c * 32, v + c * 32);
            tmem_wait_ld();
            const int j = Sh::kStreams * i + s;
            if (j >= partial) {      // (rows that are not there may see anything in the blocks before)
                const int left = limit - j * kBlockKeys;
#pragma unroll
                for (int c0 = 0; c0 < 128; c0 += 32) {
                    // a bit per key that the row sees
                    const uint32_t seen = left >= c0 + 32 ? ~0u : left <= c0 ? 0u : (1u << (left - c0)) - 1;
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!(seen & (1u << c))) v[c0 + c] = 0xff800000u;
                }
            }
            float mx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) mx[c] = fmaxf(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1]));
#pragma unroll
            for (int c = 8; c < 128; c += 2)
                mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
            const float raw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), top = raw * scale2;
            if (i == 0) {
                m = top;
                m_raw = raw;
            } else {
                const bool grow = (raw - m_raw) * scale2 > kGrow;
                if (__any_sync(~0u, grow)) {
                    // every product into O has completed: S was issued after them
                    const float f = grow ? ex2(m - top) : 1.0f;
                    if (grow) m = top, m_raw = raw;
                    l *= f;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t w[16];
                        tmem_ld16(tmem + kTmemO + s * 128 + quarter + c * 16, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
                        tmem_st16(tmem + kTmemO + s * 128 + quarter + c * 16, w);
                    }
                }
            }
            float k = scale2, base = base_of(m);
            if (far_score(base)) far_scale(m_raw, k, base);
            const uint64_t k2 = pack2(k, k), b2 = pack2(-base, -base);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t w[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const int at = q * 64 + 2 * c;
                    const float2 x = unpack2(fma2(pack2(__uint_as_float(v[at]), __uint_as_float(v[at + 1])), k2, b2));
                    const float e0 = ex2(x.x), e1 = ex2(x.y);
                    sum[c & 1] = add2(sum[c & 1], pack2(e0, e1));
                    w[c] = pack16<T>(e0, e1);
                }
                tmem_st16(sa + q * 32, w);
                tmem_st16(sa + q * 32 + 16, w + 16);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * s + q]);
            }
            const float2 x = unpack2(add2(sum[0], sum[1]));
            l += x.x + x.y;
        }
        if (mine > 0 && ok) {
            ok = warp_wait(&o_full[s], 0, timed_out);
            tc_fence_after();
        }
        // one tile on two streams: the second hands its O, four columns by row, and (m, l) to the first,
        // through the stages of the ring that were its own
        float4 *hand = reinterpret_cast<float4 *>(ring + 2 * kTile);
        float f0 = 1.0f, f1 = 0.0f;
        bool all_ok = ok;
        if (TURNS) {
            float2 *hand_ml = reinterpret_cast<float2 *>(full + 32);
            if (s == 1) {
                if (ok && mine > 0) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t w[32];
                        tmem_ld32(tmem + kTmemO + 128 + quarter + c * 32, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            hand[(c * 8 + e) * kRows + r] = make_float4(__uint_as_float(w[4 * e]), __uint_as_float(w[4 * e + 1]),
                                                                        __uint_as_float(w[4 * e + 2]), __uint_as_float(w[4 * e + 3]));
                    }
                }
                hand_ml[r] = make_float2(m, l);
            }
            asm volatile("bar.sync 2, 256;" ::: "memory");
            if (s == 0) {
                const float2 other = hand_ml[r];
                const float top = fmaxf(m, other.x), base = base_of(top);
                f0 = ex2(m - base);
                f1 = ex2(other.x - base);
                l = l * f0 + other.y * f1;
                m = top;
            }
            all_ok = ok && s == 0;
        }
        if (all_ok) {
            const int64_t row = (int64_t(me.q0) + t) * J.q_heads + int64_t(h) * A.G + g;
            const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
            const bool extra = *reinterpret_cast<volatile uint32_t *>(odd) != 0, wide = J.out_dtype == TRIT_F32;
            // The rows go out through the warp's part of the queries' tile (every S has completed): D 16-bit
            // columns of each, or D / 2 of 32 bits, whose 16-byte pieces lie so that neither way of
            // going through them meets a bank twice.
            constexpr int kChunks = D / 8;
            uint4 *stage = reinterpret_cast<uint4 *>(qs + (warp & 3) * (kTile / 4));
            auto stage_at = [&](int rl, int ch) { return stage + rl * kChunks + (ch ^ (rl & (kChunks - 1))); };
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t w[32];
                if (mine > 0) {
                    tmem_ld32(tmem + kTmemO + s * 128 + quarter + c * 32, w);
                    tmem_wait_ld();
                }
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = limit > 0 ? __uint_as_float(w[e]) * (TURNS ? f0 * inv : inv) : 0.0f;
                if (TURNS && n1 > 0 && limit > 0) {
                    const float f = f1 * inv;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 o1 = hand[(c * 8 + e) * kRows + r];
                        y[4 * e] = fmaf(o1.x, f, y[4 * e]);
                        y[4 * e + 1] = fmaf(o1.y, f, y[4 * e + 1]);
                        y[4 * e + 2] = fmaf(o1.z, f, y[4 * e + 2]);
                        y[4 * e + 3] = fmaf(o1.w, f, y[4 * e + 3]);
                    }
                }
                if (extra && there) {      // what was taken out of V and the row does see
                    for (int j = partial * kBlockKeys; j < limit; ++j) {
                        const T *v = static_cast<const T *>(J.v) + (int64_t(me.k0) + j) * J.v_stride + h * D + c * 32;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const uint32_t x = __ldg(reinterpret_cast<const uint32_t *>(v + e));
                            const float2 f = unpack16<T>(x);
                            if ((x & 0x7fffu) >= inf_bits<T>()) y[e] += f.x;
                            if (((x >> 16) & 0x7fffu) >= inf_bits<T>()) y[e + 1] += f.y;
                        }
                    }
                }
                if (wide) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *stage_at(lane, (c * 8 + e) % kChunks) =
                            make_uint4(__float_as_uint(y[4 * e]), __float_as_uint(y[4 * e + 1]), __float_as_uint(y[4 * e + 2]),
                                       __float_as_uint(y[4 * e + 3]));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *stage_at(lane, c * 4 + e) =
                            make_uint4(pack16<T>(y[8 * e], y[8 * e + 1]), pack16<T>(y[8 * e + 2], y[8 * e + 3]),
                                       pack16<T>(y[8 * e + 4], y[8 * e + 5]), pack16<T>(y[8 * e + 6], y[8 * e + 7]));
                }
                // a full stage: whole rows of it go out, a row's pieces by neighbouring lanes
                if (wide ? (c * 8 + 8) % kChunks == 0 : c + 1 == D / 32) {
                    __syncwarp();
                    const int64_t row_bytes = wide ? D * 4 : D * 2, first = wide ? (c * 8 / kChunks) * (D * 2) : 0;
#pragma unroll
                    for (int k = 0; k < kChunks; ++k) {
                        const int rl = k * (32 / kChunks) + lane / kChunks, ch = lane % kChunks;
                        const int64_t to = __shfl_sync(~0u, there ? row : int64_t(-1), rl);
                        if (to >= 0)
                            *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(J.out) + to * row_bytes + first + ch * 16) =
                                *stage_at(rl, ch);
                    }
                    __syncwarp();
                }
            }
            if (J.lse && there) J.lse[row] = lse_of(m, l);
        }
    }
    if (*reinterpret_cast<volatile uint32_t *>(timed_out)) {
        // a wait gave up: copies and products still in flight land in microseconds; give
        // them 2 ms before this CTA's memory is anyone else's
        const unsigned long long from = global_ns();
        while (global_ns() - from < 2000000ull) __nanosleep(1000);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *timed_out) raise_flag(A.err, TRIT_ERR_TIMEOUT);
    if (warp == kMmaWarp) {
        tc_fence_after();
        free_tmem();
    }
}

// Rows of `heads` vectors as (column, head, row); a copy is 64 columns of `box_heads` heads
// of `box_rows` rows.
bool make_map(CUtensorMap *map, const trit_prompt_job &J, const void *base, int heads, int64_t rows, int64_t stride,
              int box_heads, int box_rows) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {cuuint64_t(J.head_dim), cuuint64_t(heads), cuuint64_t(rows)};
    const cuuint64_t strides[2] = {cuuint64_t(J.head_dim) * 2, cuuint64_t(stride) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_rows)};
    const cuuint32_t unit[3] = {1, 1, 1};
    return fn(map, J.dtype == TRIT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void *>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, bool TURNS>
cudaError_t launch(const PromptArgs &A, int64_t grid, cudaStream_t s) {
    const trit_prompt_job &J = A.J;
    CUtensorMap qmap, kmap, vmap;
    // (without keys nothing is loaded: the maps may describe anything)
    const bool none = J.k_rows == 0;
    if (!make_map(&qmap, J, J.q, J.q_heads, J.q_rows, J.q_stride, A.heads, A.unit) ||
        !make_map(&kmap, J, none ? J.q : J.k, J.heads, none ? 1 : J.k_rows, none ? J.q_stride : J.k_stride, 1, kBlockKeys) ||
        !make_map(&vmap, J, none ? J.q : J.v, J.heads, none ? 1 : J.k_rows, none ? J.q_stride : J.v_stride, 1, kBlockKeys))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(prompt_kernel<T, D, TURNS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(Shape<D, TURNS>::kSmem));
    if (e != cudaSuccess) return e;
    // the register split draws on what the launch allocates: never start it with less
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, prompt_kernel<T, D, TURNS>);
    if (e != cudaSuccess) return e;
    if (f.numRegs != Shape<D, TURNS>::kLaunchRegs) return cudaErrorInvalidDeviceFunction;
    return launch_pdl(prompt_kernel<T, D, TURNS>, dim3(unsigned(grid)), dim3(Shape<D, TURNS>::kThreads),
                      Shape<D, TURNS>::kSmem, s, A, qmap, kmap, vmap);
}

template <typename T, int D>
cudaError_t launch_d(const PromptArgs &A, bool turns, int64_t grid, cudaStream_t s) {
    return turns ? launch<T, D, true>(A, grid, s) : launch<T, D, false>(A, grid, s);
}
template <typename T>
cudaError_t launch_t(const PromptArgs &A, bool turns, int64_t grid, cudaStream_t s) {
    return A.J.head_dim == 128 ? launch_d<T, 128>(A, turns, grid, s) : launch_d<T, 64>(A, turns, grid, s);
}

}  // namespace
}  // namespace attn

cudaError_t launch_attn_prompt(const trit_prompt_job &J, uint32_t *err, cudaStream_t s) {
    attn::PromptArgs A;
    A.J = J;
    A.err = err;
    A.scale2 = J.scale * 1.4426950408889634f;
    A.G = J.q_heads / J.heads;
    A.heads = A.G < attn::kRows ? A.G : attn::kRows;
    A.unit = attn::kRows / A.heads;
    A.parts = (A.G + attn::kRows - 1) / attn::kRows;
    A.page = A.parts * J.heads;
    // tiles: at most one begun for each sequence (whose rows are apart: keep_apart)
    const int64_t sms = device_sm_count(), grid = (J.q_rows / A.unit + J.B) * A.page;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    const bool turns = grid <= sms;
    // The search for the next longest pays where an SM takes a few tiles: four prompts of 595 to 1003
    // tokens behind 4125 to 9000 keys (512 tiles) 187 us, in their order 211; sixteen of 129 to 2048
    // (2800 tiles) 164 and 154.  Where between the two the orders cross has not been measured.
    A.sorted = J.B > 1 && J.B <= 32 && grid <= 4 * sms;
    return J.dtype == TRIT_BF16 ? attn::launch_t<__nv_bfloat16>(A, turns, grid, s) : attn::launch_t<__half>(A, turns, grid, s);
}

}  // namespace trit
