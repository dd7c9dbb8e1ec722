// The shared prefix of trit_attn_paged on the 5th-generation tensor cores: all
// rows of the batch that read key head h -- B T Hq/Hkv of them -- against the
// prefix's keys, read once per 256 rows.
//
// With R rows to a key the work is 4 D R flops on 4 D bytes, so above a few
// hundred rows the tensor cores bound it, and before them the exponentials: 128 keys
// x 128 rows take 2 x 512 SM-clocks of tensor pipe (S = Q K^T, then O += P V)
// and 16384 exponentials.  One CTA therefore runs two streams, each a
// 128-row softmax (one row per thread, no shuffles) on its own warpgroup and its
// own accumulators in tensor memory, so that one stream's products run under
// the other's softmax: S (128 x 128 fp32), overwritten in place by P (16-bit,
// the A operand of the second product, which reads it from tensor memory), and
// O (128 x D fp32).  Two row tiles of a head share the loads of K and V as the
// two streams; a single tile's streams take alternate blocks of 128 keys.
//
// K and V blocks come page by page through TMA (128-byte swizzle) into a ring.
// V is read as stored, keys by columns: an MN-major B operand.  O is rescaled
// only when a row's maximum grew by more than 2^8 since its base was fixed; until
// then P may exceed 1 (at most 2^8) and both l and O carry the same base.
//
// Each item (256 or 128 rows of a head) is cut along the keys into parts, one CTA
// each, as many as prefix_layout finds best beside the sequences' own keys; the partial results (unnormalised O, base, l) are joined with the
// sequences' own by the join kernel.  They are stored four columns by row,
// [D/4][128] float4, so that a warp's 32 rows store 512 contiguous bytes.
//
// Measured: 1024 rows of D = 128 on each of 5 heads against 32768 keys, on 80 of 152 SMs,
// beside the sequences' own keys: 137 us in all, 645 TFLOP/s, most of it here; what bounds
// it is the chain of a stream's block (S, softmax, P V, S).  P goes to the products in
// quarters of 32 keys (in halves: 151 us).
#include <cuda.h>

#include "trit_attn.cuh"
#include "trit_tc.cuh"

namespace trit {
namespace attn {
namespace {

using namespace tc;

constexpr int kBlockKeys = 128;
constexpr int kRows = 128;
constexpr int kRing = 4;
constexpr int kMmaWarp = 8;       // 8 and 9: an issuing warp per stream
constexpr int kLoadWarp = 10;     // 10 and 11: K's copies and V's
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

template <typename T>
__host__ __device__ constexpr uint32_t type_bits() { return 0; }
template <>
__host__ __device__ constexpr uint32_t type_bits<__nv_bfloat16>() { return (1u << 7) | (1u << 10); }

// Instruction descriptors, kind::f16, fp32 accumulator, M = 128: S (N = 128, both
// operands K-major) and O (N = D, B MN-major).
template <typename T>
__host__ __device__ constexpr uint32_t idesc_s() { return (1u << 4) | type_bits<T>() | ((128u >> 3) << 17) | ((128u >> 4) << 24); }
template <typename T, int D>
__host__ __device__ constexpr uint32_t idesc_o() {
    return (1u << 4) | type_bits<T>() | (1u << 16) | ((uint32_t(D) >> 3) << 17) | ((128u >> 4) << 24);
}

// Shared-memory matrix descriptors as two words: the start address and leading
// offset, and the stride (1024 bytes between groups of eight 128-byte rows),
// version and 128-byte swizzle.  A step along the operand adds to the first word
// only.  K-major (Q, K): the leading offset is unused.  MN-major (V as stored: 64
// columns of a key contiguous, 8 keys an atom): it is the distance of the
// next 64 columns, half a tile.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescK = 1u << 16, kDescMn = uint32_t((kBlockKeys * 128) >> 4) << 16;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return saddr >> 4; }

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(uint32_t(acc)), "r"(kDescHi));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n mov.b64 b, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(uint32_t(acc)), "r"(kDescHi));
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

// Waits for the phase of the given parity; false once *timed_out is set or kWaitNs
// have passed.  The clock is read every 256 tries only: a read of it
// takes longer than the waits here.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, uint32_t *timed_out) {
    unsigned long long t0 = 0;
    for (uint32_t i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 255) == 255) {
            if (*reinterpret_cast<volatile uint32_t *>(timed_out)) return false;
            const unsigned long long t = global_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitNs) {
                atomicExch(timed_out, 1u);
                return false;
            }
        }
    }
}

// Two fp32 lanes in one 64-bit register.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// The same for a whole warp: one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint32_t *timed_out) {
    return __all_sync(~0u, bar_wait(bar, parity, timed_out));
}

#define TRIT_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define TRIT_W8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])

// 32 consecutive columns of the warp's 32 tensor-memory lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : TRIT_R8(v, 0), TRIT_R8(v, 8), TRIT_R8(v, 16), TRIT_R8(v, 24)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : TRIT_R8(v, 0), TRIT_R8(v, 8)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::
            TRIT_W8(v, 0),
        TRIT_W8(v, 8), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_page(void *dst, const CUtensorMap *map, int x, int slot, int head, int page,
                                         uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2,%3,%4,%5}], [%6];" ::
            "r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(slot), "r"(head), "r"(page), "r"(smem_u32(bar))
        : "memory");
}

// The address of the tensor memory is in shared memory: a barrier of the softmax and
// issuing warps.
__device__ __forceinline__ void tmem_ready() { asm volatile("bar.sync 1, 320;" ::: "memory"); }

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ Args A, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
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
    uint64_t *tail = q_full + 1;         // the last V block's copies, before its end is cleared
    uint64_t *go = tail + 1;             // the second stream may start
    constexpr int kBars = 2 * kRing + 17;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(go + 1);
    uint32_t *timed_out = tmem_slot + 1;

    const trit_attn_job &J = A.J;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int item = int(blockIdx.x) % A.tc_items, split = int(blockIdx.x) / A.tc_items;
    const int group = item % A.tc_groups, h = item / A.tc_groups;
    const int P = int(J.batch.prefix_len);
    const int nb = (P + kBlockKeys - 1) / kBlockKeys;
    int splits = A.tc_splits;
    if (A.tc_plans > 1) {      // the own steps decide: each warp adds them up
        pdl_wait();
        const int cap = J.batch.table_pages * J.cache.page_size;
        int64_t steps = 0;
        for (int i = lane; i < J.batch.B; i += 32) {
            int len = J.batch.lens[i];
            len = len < 0 ? 0 : (len > cap ? cap : len);
            steps += (len + A.own_step - 1) / A.own_step;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) steps += __shfl_xor_sync(~0u, steps, o);
        splits = splits_of(A, steps * J.cache.heads * A.own_tiles);
        if (split >= splits) return;
    }
    const int j0 = int(int64_t(nb) * split / splits), j1 = int(int64_t(nb) * (split + 1) / splits);
    const int n = j1 - j0;
    const bool pair = 2 * group + 1 < A.tc_tiles;     // two row tiles, or one over two streams

    if (warp == kMmaWarp && lane < kBars) {       // a barrier per lane, in the order above
        const int i = lane;
        const int count = i < kRing ? 1 : i < 2 * kRing ? (pair ? 2 : 1)     // empty: streams that read the tile
                        : i < 2 * kRing + 2 ? 1 : i < 2 * kRing + 10 ? 4      // s_full, p_full (warps)
                        : i < 2 * kRing + 14 ? 1 : i == 2 * kRing + 14 ? 8 : 1;   // o_full and pv_done, q_full (warps), tail, go
        mbar_init(full + i, uint32_t(count));
        if (i == 0) *timed_out = 0;
        fence_barrier_init();
    }
    if (warp == kLoadWarp && lane < 2)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &vmap : &kmap) : "memory");
    __syncthreads();
    // the kernels behind this one start once every CTA has passed here, and rely on it
    // for all that came before
    pdl_wait();
    pdl_launch();

    // A block's place in the ring's order of use: K0 V0 K1 V1 ... for a pair, K0 K1 V0 K2 V1 ...
    // for one tile on two streams.  A wait by parity is sound only if the use before it on
    // the same stage has completed for the waiter: for a pair both streams consume every
    // tile; for one tile every stage serves one stream (K of odd blocks 1, of even ones 3, V
    // of odd blocks 0, of even ones 2) but for K0, which the second stream waits for before it
    // starts.  (The last V keeps its place behind a K that is not there.)  That wait is on a
    // barrier of its own, which completes once: the first stream's barriers go on without the
    // second, and a phase that it did not look at in time would not come again.
    auto k_at = [&](int j) { return pair ? 2 * j : (j == 0 ? 0 : 2 * j - 1); };
    auto v_at = [&](int j) { return pair ? 2 * j + 1 : 2 * j + 2; };

    // every warp of a warpgroup gives up or takes the same number of registers
    if (warp >= kLoadWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const int ps = J.cache.page_size;
        const int rows = ps < kBlockKeys ? ps : kBlockKeys;      // keys of one copy
        const int npages = (P + ps - 1) / ps;
        // page ids, 32 at a time: lane i holds the page of copy `have + i` of this CTA's keys,
        // and the next 32 are on their way
        const int per_block = kBlockKeys / rows;
        const int first_page = ps <= kBlockKeys ? j0 * per_block : 0;
        auto fetch = [&](int copy) {      // the page of this CTA's copy `copy`
            const int i = ps <= kBlockKeys ? first_page + copy : (j0 + copy) / (ps / kBlockKeys);
            return i < npages ? __ldg(J.batch.prefix_table + i) : -1;
        };
        int have = 0, ids = fetch(lane), ids_next = fetch(32 + lane);
        const bool is_v = warp > kLoadWarp;
        const CUtensorMap *map = is_v ? &vmap : &kmap;
        const int c = lane / (D / 64), half = lane % (D / 64);     // the lane's copy of a block
        for (int j = 0; j < n; ++j) {
            const int at = is_v ? v_at(j) : k_at(j), s = at % kRing;
            const int key0 = (j0 + j) * kBlockKeys;
            const int first = key0 / ps;
            const int copies = per_block < npages - first ? per_block : npages - first;
            const int keys = P - key0 < kBlockKeys ? P - key0 : kBlockKeys;
            const bool clear = is_v && keys < kBlockKeys;
            uint64_t *bar = clear ? tail : &full[s];
            uint8_t *st = ring + s * kTile;
            if (j * per_block >= have + 32) {
                have += 32;
                ids = ids_next;
                ids_next = fetch(have + 32 + lane);
            }
            const int page = __shfl_sync(~0u, ids, (j * per_block + c - have) & 31);
            if (c < copies && (page < 0 || page >= J.cache.pages)) raise_flag(A.err, TRIT_ERR_INDEX);   // reads as zeros
            if (!warp_wait(&empty[s], ((at / kRing) & 1) ^ 1, timed_out)) break;
            if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(copies) * rows * D * 2);
            __syncwarp();
            if (c < copies)
                tma_page(st + half * (kBlockKeys * 128) + c * rows * 128, map, half * 64, key0 - first * ps, h, page, bar);
            if (clear) {   // keys past the prefix get P = 0, which must not meet a NaN
                if (!warp_wait(tail, 0, timed_out)) break;
                for (int i = lane; i < (kBlockKeys - keys) * (D / 8); i += 32) {
                    const int r = keys + i / (D / 8), ch = i % (D / 8);
                    *reinterpret_cast<uint4 *>(st + (ch / 8) * (kBlockKeys * 128) + r * 128 + (ch % 8) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
            }
        }
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
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
        const int s = warp - kMmaWarp, mine = pair ? n : (n + 1 - s) / 2;
        const bool leader = elect_one();
        const uint32_t qlo = (desc_lo(smem_u32(qs)) | kDescK) + (pair ? s * (kTile >> 4) : 0);
        const uint32_t rk = desc_lo(smem_u32(ring)) | kDescK, rv = desc_lo(smem_u32(ring)) | kDescMn;
        const uint32_t sp = tmem + s * 128, o = tmem + 256 + s * 128;
        auto k_there = [&](int i) -> bool {
            const int at = k_at(pair ? i : 2 * i + s);
            return warp_wait(&full[at % kRing], (at / kRing) & 1, timed_out);
        };
        auto issue_s = [&](int i) {
            const int st = k_at(pair ? i : 2 * i + s) % kRing;
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
        bool ok = warp_wait(q_full, 0, timed_out);
        // the streams start half a block apart: in step, they would want the tensor
        // pipe together and then the exponentials together (measured: 4100 SM-clocks a
        // block pair in step): with the first stream's second block, or behind its first where
        // there are few
        const int go_block = n >= 8 ? 1 : 0, go_part = n >= 8 ? 0 : 3;
        if (s == 1) ok = ok && warp_wait(go, 0, timed_out);
        if (ok && mine > 0) {
            ok = k_there(0);
            if (ok) issue_s(0);
        }
        for (int i = 0; ok && i < mine; ++i) {
            const int at = v_at(pair ? i : 2 * i + s), st = at % kRing;
            ok = warp_wait(&full[st], (at / kRing) & 1, timed_out);
            const uint32_t b = rv + st * (kTile >> 4);
#pragma unroll
            for (int part = 0; part < 4; ++part) {
                ok = ok && warp_wait(&p_full[4 * s + part], i & 1, timed_out);
                if (!ok) break;
                if (s == 0 && i == go_block && part == go_part && lane == 0) mbar_arrive(go);
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 2 * part; kk < 2 * part + 2; ++kk)
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
                ok = k_there(i + 1) && warp_wait(&pv_done[s], i & 1, timed_out);
                if (ok) issue_s(i + 1);
            }
        }
    } else {
        // softmax: stream s, row r of its tile (tensor-memory lane r)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int s = warp >> 2, r = threadIdx.x & 127;
        const uint32_t quarter = uint32_t((warp & 3) * 32) << 16;
        {   // the query tile: every lane finds one row, then the warp copies whole rows
            constexpr int CH = D / 8, RI = 32 / CH;
            const int tile = 2 * group + (pair ? s : 0);
            uint8_t *dst = qs + (pair ? s * kTile : 0);
            const int fr = tile * kRows + r, rows = J.batch.B * A.R;
            const int b = fr / A.R, rr = fr - b * A.R, t = rr / A.G, g = rr - t * A.G;
            const int64_t mine_at = fr < rows ? (int64_t(b) * J.batch.T + t) * J.q_stride + (int64_t(h) * A.G + g) * D : -1;
            const int c = lane % CH;
            uint4 v[CH];
#pragma unroll
            for (int j = 0; j < CH; ++j) {       // every load before the first store: one latency
                // (rows that are not there read row 0, without a branch that would wait for each load)
                const int64_t at = __shfl_sync(~0u, mine_at, j * RI + lane / CH);
                v[j] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(J.q) + (at < 0 ? 0 : at)) + c);
            }
#pragma unroll
            for (int j = 0; j < CH; ++j) {       // 32 rows, RI at a time (of a shared tile each stream takes half)
                if (!pair && (j >= CH / 2) != (s == 1)) continue;
                const int row = (warp & 3) * 32 + j * RI + lane / CH;
                const uint32_t keep = tile * kRows + row < rows ? A.keep : 0u;
                v[j].x = (v[j].x & keep) ^ A.flip; v[j].y = (v[j].y & keep) ^ A.flip;
                v[j].z = (v[j].z & keep) ^ A.flip; v[j].w = (v[j].w & keep) ^ A.flip;
                *reinterpret_cast<uint4 *>(dst + (c / 8) * (kRows * 128) + sw128_off(row, c % 8)) = v[j];
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        tmem_ready();     // after the queries: the allocation takes as long
        tc_fence_after();
        const uint32_t tmem = *tmem_slot;
        const float scale2 = A.scale2;
        const int mine = pair ? n : (n + 1 - s) / 2;       // this stream's blocks
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int i = 0; i < mine; ++i) {
            ok = warp_wait(&s_full[s], i & 1, timed_out);
            if (!ok) break;
            tc_fence_after();
            const int j = pair ? i : 2 * i + s;
            const int left = P - (j0 + j) * kBlockKeys;
            const uint32_t sa = tmem + s * 128 + quarter;
            uint32_t v[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(sa + c * 32, v + c * 32);
            tmem_wait_ld();
            if (left < kBlockKeys) {
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
                    const float2 t = unpack2(fma2(pack2(__uint_as_float(v[at]), __uint_as_float(v[at + 1])), k2, b2));
                    const float e0 = ex2(t.x), e1 = ex2(t.y);
                    sum[c & 1] = add2(sum[c & 1], pack2(e0, e1));
                    w[c] = pack16<T>(e0, e1);
                }
                tmem_st16(sa + q * 16, w);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[4 * s + q]);
            }
            const float2 t = unpack2(add2(sum[0], sum[1]));
            l += t.x + t.y;
        }
        float *part = A.tc_parts + ((int64_t(item) * A.tc_splits + split) * 2 + s) * part_floats(kRows, D);
        if (mine > 0 && ok) {
            ok = warp_wait(&o_full[s], 0, timed_out);
            tc_fence_after();
            if (ok) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t w[32];
                    tmem_ld32(tmem + 256 + s * 128 + quarter + c * 32, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<uint4 *>(part + ((c * 8 + e) * kRows + r) * 4) =
                            make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                }
            }
        }
        *reinterpret_cast<float2 *>(part + kRows * D + 2 * r) = make_float2(m, l);
    }
    if (*reinterpret_cast<volatile uint32_t *>(timed_out)) {
        // a wait gave up: copies and products still in flight land in microseconds; give
        // them 2 ms before this CTA's memory is anyone else's
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < 2000000ull) __nanosleep(1000);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *timed_out) raise_flag(A.err, TRIT_ERR_TIMEOUT);
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tmem_slot), "r"(kTmemCols));
    }
}

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// The cache as (column, slot, head, page); a copy is 64 columns of min(page_size,
// 128) keys of one head's page.
bool make_map(CUtensorMap *map, const trit_kv_cache &C, void *base) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[4] = {cuuint64_t(C.head_dim), cuuint64_t(C.page_size), cuuint64_t(C.heads),
                                cuuint64_t(C.pages)};
    const cuuint64_t one = cuuint64_t(C.head_dim) * 2;   // a dimension of one entry needs no stride
    const cuuint64_t strides[3] = {C.page_size > 1 ? cuuint64_t(C.slot_stride) * 2 : one,
                                   C.heads > 1 ? cuuint64_t(C.head_stride) * 2 : one,
                                   C.pages > 1 ? cuuint64_t(C.page_stride) * 2 : one};
    const cuuint32_t box[4] = {64, cuuint32_t(C.page_size < kBlockKeys ? C.page_size : kBlockKeys), 1, 1};
    const cuuint32_t unit[4] = {1, 1, 1, 1};
    return fn(map, C.dtype == TRIT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base,
              dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch(const Args &A, cudaStream_t s) {
    CUtensorMap kmap, vmap;
    if (!make_map(&kmap, A.J.cache, A.J.cache.k) || !make_map(&vmap, A.J.cache, A.J.cache.v))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(prefix_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(smem_bytes<D>()));
    if (e != cudaSuccess) return e;
    // the register split draws on what the launch allocates: never start it with less
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, prefix_kernel<T, D>);
    if (e != cudaSuccess) return e;
    if (f.numRegs != kLaunchRegs) return cudaErrorInvalidDeviceFunction;
    return launch_pdl(prefix_kernel<T, D>, dim3(unsigned(A.tc_items * A.tc_splits)), dim3(kThreads), smem_bytes<D>(), s, A,
                      kmap, vmap);
}

}  // namespace

bool prefix_on_tensor_cores(const trit_attn_job &J) {
    const trit_kv_cache &C = J.cache;
    const int64_t rows = int64_t(J.batch.B) * J.batch.T * (J.q_heads / C.heads);
    const bool pow2 = (C.page_size & (C.page_size - 1)) == 0;
    // strides a copy's descriptor cannot hold (or that overlap) stay on the other path
    const int64_t most = int64_t(1) << 38;
    const bool strides = C.slot_stride >= C.head_dim && (C.heads == 1 || C.head_stride >= C.head_dim) &&
                         (C.pages == 1 || C.page_stride >= C.head_dim) && C.slot_stride < most &&
                         C.head_stride < most && C.page_stride < most;
    // From 17 rows: 20 rows behind 4096 and 32768 keys 16.3 and 32.4 us here, 21.0 and 34.6 on the
    // other path; 32 rows 17.5 and 33.5 against 18.4 and 41.6; 64 rows 19.8 and 36.2 against
    // 26.5 and 54.7 (in all, 33 to 900 own keys).  Fewer leave most of 128 lanes empty.
    return J.batch.prefix_len > 0 && rows > 16 && pow2 && C.page_size >= 16 && strides;
}

void prefix_layout(Args &A, int64_t most) {
    const trit_attn_job &J = A.J;
    const int64_t rows = int64_t(J.batch.B) * A.R;
    const int nb = int((J.batch.prefix_len + kBlockKeys - 1) / kBlockKeys);
    A.tc_tiles = int((rows + kRows - 1) / kRows);
    A.tc_groups = (A.tc_tiles + 1) / 2;
    A.tc_items = A.tc_groups * J.cache.heads;
    // The parts s each item is cut into, by a model in us fitted to sweeps.  The prefix
    // kernel's items * s CTAs take an SM each: 4 us and, per block of 128 keys, 1.6 for a
    // pair of tiles (1.3 where D = 64) or 1.2 for one (0.9).  The own-keys kernel's CTAs
    // beside it: 8 us and 1.25 per step (1.43 where D = 64, 2.2 for more than 16 rows).
    // Every part is written and read once more.  (2.0 and 1.6, or 1.4 and 1.1, per block
    // choose parts that take 41.4 instead of 39.8 us for 24 x 5 drafts and 41.7 or 44.4 instead of
    // 39.6 for 96 sequences of D = 64.  256 sequences behind 32768 keys, before P went in
    // quarters, 3, 4, 5 parts: 196, 151, 165.)
    const bool single = A.tc_tiles == 1, wide = J.cache.head_dim == 128;
    const double per_block = wide ? (single ? 1.2 : 1.6) : (single ? 0.9 : 1.3);
    const double per_step = A.RT > 16 ? 2.2 : wide ? 1.25 : 1.43;
    const double per_split = double(rows) * J.cache.heads * J.cache.head_dim * 4 / 5e6 * (single ? 2 : 1);
    // (this runs in every call: the terms without W once, then a few operations each)
    constexpr int kMost = 64;
    double prefix[kMost + 1], per_own[kMost + 1];
    int top = 0;
    for (int s = 1; s <= nb && s <= kMost && (s == 1 || s * A.tc_items <= kSms - 8); ++s) {
        const int ctas = s * A.tc_items, waves = (ctas + kSms - 1) / kSms;
        const int beside = kSms - ctas > 8 ? kSms - ctas : 8;
        prefix[s] = waves * (4 + (nb + s - 1) / s * per_block);
        per_own[s] = per_step / (double(beside) * A.resident);
        top = s;
    }
    auto cost = [&](int s, double W) {
        const double floor = per_step * (W < 4 * kSms ? W / kSms : 4);    // chunks are not cut shorter
        double own = W * per_own[s];
        own = 8 + (own > floor ? own : floor);
        return (prefix[s] > own ? prefix[s] : own) + s * per_split;
    };
    auto best = [&](double W) {
        int parts = 1;
        for (int s = 2; s <= top; ++s)
            if (cost(s, W) < cost(parts, W)) parts = s;
        return parts;
    };
    const double widest = 1.25 * double(most);
    const int half = best(double(most) / 2);      // for half of the tables' room
    // fewer parts as the own steps grow: the steps from which each number is best, or one
    // number where that costs no more than 4 us at either end (adding the steps up, and CTAs
    // that then have no part, cost 1.5)
    const bool one = cost(half, 0) < cost(best(0), 0) + 4 && cost(half, widest) < cost(best(widest), widest) + 4;
    A.tc_plans = 1;
    A.tc_parts_for[0] = A.tc_splits = one ? half : best(0);
    A.tc_from[0] = 0;
    for (double W = 256; !one && W < widest && A.tc_plans < kPlans; W *= 1.3) {
        const int s = best(W);
        if (s == A.tc_parts_for[A.tc_plans - 1]) continue;
        A.tc_parts_for[A.tc_plans] = s;
        A.tc_from[A.tc_plans++] = int64_t(W);
        if (s > A.tc_splits) A.tc_splits = s;
    }
    // the own-keys kernel's grid: what fits beside those parts (a CTA without a chunk would
    // run last, on an SM it has to wait for)
    const int64_t fit = int64_t(kSms - A.tc_items * half) * A.resident;
    if (fit >= kSms && fit < A.grid) A.grid = int(fit);
}

cudaError_t launch_prefix(const Args &A, cudaStream_t s) {
    if (A.J.cache.dtype == TRIT_BF16)
        return A.J.cache.head_dim == 128 ? launch<__nv_bfloat16, 128>(A, s) : launch<__nv_bfloat16, 64>(A, s);
    return A.J.cache.head_dim == 128 ? launch<__half, 128>(A, s) : launch<__half, 64>(A, s);
}

int64_t prefix_part_bytes(const Args &A) {
    return int64_t(A.tc_items) * A.tc_splits * 2 * part_floats(kRows, A.J.cache.head_dim) * 4;
}

}  // namespace attn
}  // namespace trit
