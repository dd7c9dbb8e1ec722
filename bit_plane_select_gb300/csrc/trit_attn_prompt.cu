// trit_attn_prompt: causal attention of packed prompts on the 5th-generation tensor
// cores.
//
// With n queries 4 D Hq flops a pair of query and key on 2 D (2 Hq + 2 Hkv) bytes a token, prompts
// of more than a few hundred tokens are bound by the tensor pipe, and beside it by the
// exponentials.  As in trit_attn_prefix.cu a CTA runs two streams, each a 128-row
// softmax (one row per thread, no shuffles) with its own S (128 x 128 fp32, overwritten
// in place by P, the 16-bit operand of the second product) and O in tensor
// memory, so that one stream's products run under the other's softmax.
//
// A row is a token and one of the G query heads that share a key head: 128 / G tokens'
// rows fill a tile, so one K and V tile serves them all, a prompt's diagonal cuts off little
// (a tile of G = 4 covers 32 tokens), and short prompts leave few rows empty.  Q, K and V
// come by TMA; the box (64 columns, G heads, 128 / G tokens) lays Q out in that order.
// The two streams take neighbouring tiles and share the loads of K and V.
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
constexpr int kRing = 4;
constexpr int kMmaWarp = 8;       // 8 and 9: an issuing warp per stream
constexpr int kLoadWarp = 10;     // 10 and 11: Q's and K's copies, and V's
constexpr int kThreads = 384;      // 8 softmax warps and the four above
// Registers: launched with 168 a thread; the softmax warpgroups, which hold a row of
// S, take 216 and the third keeps 72 (256 * 216 + 128 * 72 = 384 * 168).
constexpr int kLaunchRegs = 168;
constexpr int kTmemCols = 512;     // S of the two streams at 0 and 128, O at 256 and 384
constexpr float kGrow = 8.0f;      // log2 of the growth of a maximum that O tolerates

template <int D>
__host__ __device__ constexpr int tile_bytes() { return kBlockKeys * D * 2; }
template <int D>
constexpr size_t smem_bytes() { return 1024 + size_t(2 + kRing) * tile_bytes<D>() + 256; }

struct PromptArgs {
    trit_prompt_job J;
    uint32_t *err;
    float scale2;            // scale log2(e)
    int32_t G;               // query heads per key head
    int32_t heads;           // of a tile: min(G, 128)
    int32_t tokens;          // of a tile: 128 / heads
    int32_t parts;           // tiles that the G heads of a key head take
    int32_t page;            // parts * key heads: items of a pair of tiles' tokens
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

__device__ __forceinline__ void tma_rows(void *dst, const CUtensorMap *map, int x, int head, int row, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2,%3,%4}], [%5];" ::
            "r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(head), "r"(row), "r"(smem_u32(bar))
        : "memory");
}
// The address of the tensor memory is in shared memory: a barrier of the softmax and
// issuing warps.
__device__ __forceinline__ void tmem_ready() { asm volatile("bar.sync 1, 320;" ::: "memory"); }

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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ PromptArgs A, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int kTile = tile_bytes<D>();
    uint8_t *qs = smem, *ring = smem + 2 * kTile;
    uint64_t *full = reinterpret_cast<uint64_t *>(ring + kRing * kTile);
    uint64_t *empty = full + kRing;
    uint64_t *s_full = empty + kRing;    // stream's S is in tensor memory
    uint64_t *p_full = s_full + 2;       // [stream][quarter]: P of 32 keys each is
    uint64_t *o_full = p_full + 8;       // stream's O is finished
    uint64_t *pv_done = o_full + 2;      // stream's product into O has completed
    uint64_t *q_full = pv_done + 2;
    uint64_t *tail = q_full + 1;         // the copies of a V block that is looked through
    uint64_t *go = tail + 1;             // the second stream may start
    constexpr int kBars = 2 * kRing + 17;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(go + 1);
    uint32_t *timed_out = tmem_slot + 1;
    uint32_t *odd = tmem_slot + 2;       // V held an infinity or NaN in a block that is masked

    const trit_prompt_job &J = A.J;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kMmaWarp && lane < kBars) {       // a barrier per lane, in the order above
        const int i = lane;
        const int count = i < kRing ? 1 : i < 2 * kRing ? 2                  // empty: both streams
                        : i < 2 * kRing + 2 ? 1 : i < 2 * kRing + 10 ? 4 : 1;     // s_full, p_full (warps), the others
        mbar_init(full + i, uint32_t(count));
        if (i == 0) *timed_out = *odd = 0;
        fence_barrier_init();
    }
    if (warp == kLoadWarp && lane < 3)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap) : "memory");
    __syncthreads();
    pdl_wait();
    pdl_launch();

    // the item: a pair of tiles of one sequence (the last of a sequence first) and a key head
    const int pair_tokens = 2 * A.tokens;
    int64_t k = blockIdx.x / A.page;
    const int item = int(blockIdx.x - k * A.page), h = item / A.parts, part = item - h * A.parts;
    Span me{0, 0, 0, 0};
    int mine_pairs = 0;
    for (int b0 = 0; b0 < J.B; b0 += 32) {        // every warp for itself: 32 sequences at a time
        bool bad = false;
        Span s{0, 0, 0, 0};
        if (b0 + lane < J.B) s = span_of(A, b0 + lane, &bad);
        if (bad && blockIdx.x == 0 && warp == 0) raise_flag(A.err, TRIT_ERR_INDEX);
        const int pairs = (s.nq + pair_tokens - 1) / pair_tokens;
        int inc = pairs;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += v;
        }
        const int all = __shfl_sync(~0u, inc, 31);
        if (mine_pairs == 0 && k < all) {
            const int who = __ffs(int(__ballot_sync(~0u, k < inc))) - 1;
            me.q0 = __shfl_sync(~0u, s.q0, who);
            me.nq = __shfl_sync(~0u, s.nq, who);
            me.k0 = __shfl_sync(~0u, s.k0, who);
            me.nk = __shfl_sync(~0u, s.nk, who);
            mine_pairs = __shfl_sync(~0u, pairs, who);
            k -= __shfl_sync(~0u, inc, who) - mine_pairs;
            if (blockIdx.x) break;                // the first CTA looks at all starts
        }
        if (mine_pairs == 0) k -= all;
    }
    if (mine_pairs == 0) return;                  // more CTAs than pairs: the same for every warp
    const int t0 = int(mine_pairs - 1 - k) * pair_tokens;      // the item's first token
    const int behind = me.nk - me.nq;             // query t sees keys 0 .. t + behind
    // blocks of the streams: up to the last token's limit
    auto blocks_of = [&](int s) {
        const int from = t0 + s * A.tokens, to = min(from + A.tokens, me.nq);
        const int last = from < me.nq ? to + behind : 0;
        return last > 0 ? (last + kBlockKeys - 1) / kBlockKeys : 0;
    };
    const int n0 = blocks_of(0), n1 = blocks_of(1), n = max(n0, n1);
    const int first_limit = max(0, behind + t0 + 1);
    const int partial = first_limit / kBlockKeys;              // blocks from here on are hidden from some row

    if (warp >= kLoadWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const bool is_v = warp > kLoadWarp;
        if (!is_v && lane == 0 && n > 0) {
            const uint32_t bytes = uint32_t(A.heads * A.tokens * 128);
            mbar_arrive_expect_tx(q_full, 2 * (D / 64) * bytes);
#pragma unroll
            for (int i = 0; i < 2 * (D / 64); ++i)
                tma_rows(qs + (i / (D / 64)) * kTile + (i % (D / 64)) * (kRows * 128), &qmap, (i % (D / 64)) * 64,
                         h * A.G + part * 128, me.q0 + t0 + (i / (D / 64)) * A.tokens, q_full);
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
                constexpr uint32_t kInf = inf_bits<T>();
                uint4 *v = reinterpret_cast<uint4 *>(st);
                bool found = false;
#pragma unroll 8
                for (int i = lane; i < kTile / 16; i += 32) {
                    uint4 x = v[i];
                    const uint32_t top = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                                  __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
                    if ((top & 0xffffu) >= kInf || (top >> 16) >= kInf) {
                        x.x = finite_pair<T>(x.x); x.y = finite_pair<T>(x.y);
                        x.z = finite_pair<T>(x.z); x.w = finite_pair<T>(x.w);
                        v[i] = x;
                        found |= j * kBlockKeys + (i % (kBlockKeys * 8)) / 8 < me.nk;
                    }
                }
                if (found) *reinterpret_cast<volatile uint32_t *>(odd) = 1;
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
            }
        }
    } else if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kMmaWarp) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(kTmemCols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
            tc_fence_before();
        }
        tmem_ready();
        tc_fence_after();
        const uint32_t tmem = *tmem_slot;
        // stream s: S of its first block, then per block O += P V and S of the next,
        // which takes the place of P once that product has completed.  The whole warp
        // walks the loop (uniform values, so the operands are in uniform registers
        // when a product is issued); one elected lane issues.
        const int s = warp - kMmaWarp, mine = s ? n1 : n0;
        const bool leader = elect_one();
        const uint32_t qlo = (desc_lo(smem_u32(qs)) | kDescK) + s * (kTile >> 4);
        const uint32_t rk = desc_lo(smem_u32(ring)) | kDescK, rv = desc_lo(smem_u32(ring)) | kDescMn;
        const uint32_t sp = tmem + s * 128, o = tmem + 256 + s * 128;
        auto tile_there = [&](int at) -> bool { return warp_wait(&full[at % kRing], (at / kRing) & 1, timed_out); };
        auto issue_s = [&](int i) {
            const int st = (2 * i) % kRing;
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
        bool ok = n == 0 || warp_wait(q_full, 0, timed_out), gone = false;
        // the streams start half a block apart: in step, they would want the tensor
        // pipe together and then the exponentials together
        const int go_block = mine >= 8 ? 1 : 0, go_part = mine >= 8 ? 0 : 3;
        if (s == 1 && mine > 0) ok = ok && warp_wait(go, 0, timed_out);
        if (ok && mine > 0) {
            ok = tile_there(0);
            if (ok) issue_s(0);
        }
        for (int i = 0; ok && i < mine; ++i) {
            const int at = 2 * i + 1, st = at % kRing;
            ok = tile_there(at);
            const uint32_t b = rv + st * (kTile >> 4);
#pragma unroll
            for (int part4 = 0; part4 < 4; ++part4) {
                ok = ok && warp_wait(&p_full[4 * s + part4], i & 1, timed_out);
                if (!ok) break;
                if (s == 0 && i == go_block && part4 == go_part) {
                    if (lane == 0) mbar_arrive(go);
                    gone = true;
                }
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 2 * part4; kk < 2 * part4 + 2; ++kk)
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
                ok = tile_there(2 * (i + 1)) && warp_wait(&pv_done[s], i & 1, timed_out);
                if (ok) issue_s(i + 1);
            }
        }
        if (s == 0 && !gone && lane == 0) mbar_arrive(go);
        // blocks that only the other stream needs
        for (int at = 2 * mine; ok && at < 2 * n; ++at) {
            ok = tile_there(at);
            if (ok && lane == 0) mbar_arrive(&empty[at % kRing]);
            __syncwarp();
        }
    } else {
        // softmax: stream s, row r of its tile (tensor-memory lane r)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int s = warp >> 2, r = threadIdx.x & 127;
        const uint32_t quarter = uint32_t((warp & 3) * 32) << 16;
        tmem_ready();
        tc_fence_after();
        const uint32_t tmem = *tmem_slot;
        const float scale2 = A.scale2;
        const int mine = s ? n1 : n0;                  // this stream's blocks
        const int tile_t = r / A.heads, g = part * 128 + r - tile_t * A.heads, t = t0 + s * A.tokens + tile_t;
        const bool there = tile_t < A.tokens && t < me.nq && g < A.G;
        const int limit = there ? max(0, t + behind + 1) : 0;       // keys that the row sees
        // blocks that every row of the stream sees whole need no mask (rows that are not there may see anything)
        const int clear = max(0, t0 + s * A.tokens + behind + 1) / kBlockKeys;
        float m = -INFINITY, l = 0.0f;
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
            if (i >= clear) {
                const int left = limit - i * kBlockKeys;
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if (c >= left) v[c] = 0xff800000u;
            }
            float mx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) mx[c] = fmaxf(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1]));
#pragma unroll
            for (int c = 8; c < 128; c += 2)
                mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale2;
            if (i == 0) {
                m = top;
            } else {
                const bool grow = top > m + kGrow;
                if (__any_sync(~0u, grow)) {
                    // every product into O has completed: S was issued after them
                    const float f = grow ? ex2(m - top) : 1.0f;
                    if (grow) m = top;
                    l *= f;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t w[16];
                        tmem_ld16(tmem + 256 + s * 128 + quarter + c * 16, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
                        tmem_st16(tmem + 256 + s * 128 + quarter + c * 16, w);
                    }
                }
            }
            const float base = base_of(m);
            const uint64_t k2 = pack2(scale2, scale2), b2 = pack2(-base, -base);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t w[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const int at = q * 32 + 2 * c;
                    const float2 x = unpack2(fma2(pack2(__uint_as_float(v[at]), __uint_as_float(v[at + 1])), k2, b2));
                    const float e0 = ex2(x.x), e1 = ex2(x.y);
                    sum[c & 1] = add2(sum[c & 1], pack2(e0, e1));
                    w[c] = pack16<T>(e0, e1);
                }
                tmem_st16(sa + q * 16, w);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[4 * s + q]);
            }
            const float2 x = unpack2(add2(sum[0], sum[1]));
            l += x.x + x.y;
        }
        if (mine > 0 && ok) {
            ok = warp_wait(&o_full[s], 0, timed_out);
            tc_fence_after();
        }
        if (ok) {
            const int64_t row = (int64_t(me.q0) + t) * J.q_heads + int64_t(h) * A.G + g;
            const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
            const bool extra = *reinterpret_cast<volatile uint32_t *>(odd) != 0;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t w[32];
                if (mine > 0) {
                    tmem_ld32(tmem + 256 + s * 128 + quarter + c * 32, w);
                    tmem_wait_ld();
                }
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = limit > 0 ? __uint_as_float(w[e]) * inv : 0.0f;
                if (!there) continue;
                if (extra) {      // what was taken out of V and the row does see
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
                if (J.out_dtype == TRIT_F32) {
                    float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(J.out) + row * D + c * 32);
#pragma unroll
                    for (int e = 0; e < 8; ++e) to[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                } else {
                    uint4 *to = reinterpret_cast<uint4 *>(static_cast<T *>(J.out) + row * D + c * 32);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        to[e] = make_uint4(pack16<T>(y[8 * e], y[8 * e + 1]), pack16<T>(y[8 * e + 2], y[8 * e + 3]),
                                           pack16<T>(y[8 * e + 4], y[8 * e + 5]), pack16<T>(y[8 * e + 6], y[8 * e + 7]));
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
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tmem_slot), "r"(kTmemCols));
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

template <typename T, int D>
cudaError_t launch(const PromptArgs &A, int64_t grid, cudaStream_t s) {
    const trit_prompt_job &J = A.J;
    CUtensorMap qmap, kmap, vmap;
    // (without keys nothing is loaded: the maps may describe anything)
    const bool none = J.k_rows == 0;
    if (!make_map(&qmap, J, J.q, J.q_heads, J.q_rows, J.q_stride, A.heads, A.tokens) ||
        !make_map(&kmap, J, none ? J.q : J.k, J.heads, none ? 1 : J.k_rows, none ? J.q_stride : J.k_stride, 1, kBlockKeys) ||
        !make_map(&vmap, J, none ? J.q : J.v, J.heads, none ? 1 : J.k_rows, none ? J.q_stride : J.v_stride, 1, kBlockKeys))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(prompt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(smem_bytes<D>()));
    if (e != cudaSuccess) return e;
    // the register split draws on what the launch allocates: never start it with less
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, prompt_kernel<T, D>);
    if (e != cudaSuccess) return e;
    if (f.numRegs != kLaunchRegs) return cudaErrorInvalidDeviceFunction;
    return launch_pdl(prompt_kernel<T, D>, dim3(unsigned(grid)), dim3(kThreads), smem_bytes<D>(), s, A, qmap, kmap, vmap);
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
    A.tokens = attn::kRows / A.heads;
    A.parts = (A.G + attn::kRows - 1) / attn::kRows;
    A.page = A.parts * J.heads;
    // pairs of tiles: at most one started for each sequence
    const int64_t grid = (J.q_rows / (2 * A.tokens) + J.B) * A.page;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    if (J.dtype == TRIT_BF16)
        return J.head_dim == 128 ? attn::launch<__nv_bfloat16, 128>(A, grid, s) : attn::launch<__nv_bfloat16, 64>(A, grid, s);
    return J.head_dim == 128 ? attn::launch<__half, 128>(A, grid, s) : attn::launch<__half, 64>(A, grid, s);
}

}  // namespace trit
