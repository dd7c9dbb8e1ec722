// Attention over a paged cache: what its kernels share -- the work's layout,
// the partial results and how they are joined.
//
// A query row's softmax over keys split in parts needs of each part only
//     m = max_j s_j,  l = sum_j 2^(s_j - m),  o = sum_j 2^(s_j - m) v_j
// (s = scale log2(e) q.k): parts a and b join as m = max(m_a, m_b),
// l = l_a 2^(m_a - m) + l_b 2^(m_b - m), o likewise; out = o / l and
// lse = m ln 2 + ln l at the end.  All of it is fp32.
#pragma once

#include "trit_serve.cuh"

namespace trit {
namespace attn {

constexpr int kSms = 152;           // the grids are cut for this many
constexpr int kPlans = 8;
constexpr int kMostCtas = 3;       // CTAs of the own-keys kernel per SM, at most
constexpr int kTcRows = 128;       // rows of a tile of the tensor-core prefix kernel

// Rows: row r = t*G + g of a (sequence, key head) pair is token t and query
// head h*G + g; a prefix row is the sequence's index times R plus r.  An item
// is a tile of RT rows of one key head against either one sequence's own keys
// ("own", (b, h, tile)) or the shared prefix ("prefix", (h, tile)).
struct Args {
    trit_attn_job J;
    uint32_t *err;
    float scale2;            // |scale| log2(e) (1 where scale is 0)
    uint32_t flip, keep;     // on pairs of q: the sign of scale, and 0 where it is 0
    int32_t G, R;            // query heads per key head; rows per (sequence, key head)
    uint32_t g_inv;          // ceil(2^32 / G) where that divides any row exactly, else 0
    int32_t RT;              // rows of an item
    int32_t own_tiles;       // row tiles per (sequence, key head)
    int32_t pre_tiles;       // row tiles of the prefix, per key head (0: no prefix item)
    int32_t pre_steps;       // steps of the prefix
    int32_t grid;            // CTAs of the own-keys kernel, a chunk of the work each at most
    int32_t resident;        // of which so many fit an SM together
    int32_t page_shift;      // log2(page_size), or -1
    uint32_t *count;         // workspace: arrivals, by an item's first chunk; zero between calls
    int32_t *cum;            // workspace: [B + 1] steps of the sequences before b
    float *parts;            // workspace: the partial results
    // the prefix on the tensor cores (tc_items = 0: its items are above, with the own ones)
    int32_t tc_tiles, tc_groups;   // 128-row tiles per key head, and pairs of them
    int32_t tc_items, tc_splits;   // (head, pair) items, and the most parts each is cut into
    int32_t tc_plans;              // parts by the own steps W: tc_parts_for[i] from tc_from[i] on
    int32_t tc_parts_for[kPlans];
    int64_t tc_from[kPlans];
    int32_t own_step;        // keys of an own step
    float *tc_parts;         // workspace: their partial results, [item][tc_splits][stream]
    int32_t split;           // its keys come as two 16-bit parts, 2 D columns a key, its queries in units of their own:
    const float *q_units;    // [B T Hq]
};

// Row r's token r / G: a high product with ceil(2^32 / G) is exact for r G < 2^32.
__device__ __forceinline__ int token_of(const Args &A, int r) {
    return A.g_inv ? int(__umulhi(uint32_t(r), A.g_inv)) : r / A.G;
}

// A partial result: RT x D sums, then RT pairs (m, l).
__host__ __device__ inline int64_t part_floats(int RT, int D) { return int64_t(RT) * (D + 2); }

// Slots of partial results: chunk c's first and last unfinished items at 2c and
// 2c + 1, then one per own item and per prefix item that lies in a single chunk.
__host__ __device__ inline int64_t slot_own(const Args &A, int b, int h, int tile) {
    return 2 * int64_t(A.grid) + (int64_t(b) * A.J.cache.heads + h) * A.own_tiles + tile;
}
__host__ __device__ inline int64_t slot_prefix(const Args &A, int h, int tile) {
    return 2 * int64_t(A.grid) + int64_t(A.J.batch.B) * A.J.cache.heads * A.own_tiles +
           int64_t(h) * A.pre_tiles + tile;
}

// Quotients here are 32-bit wherever the operands are (a 64-bit division takes
// hundreds of SM-clocks).
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return int64_t(uint32_t(a) / uint32_t(b));
    return a / b;
}

// Parts of a prefix item beside W own steps.  The prefix kernel takes whole SMs and the
// own-keys kernel the others, so that tensor work and memory traffic overlap; the
// more own steps, the fewer SMs (prefix_layout).  W is known on the device only, and every
// kernel decides alike.
__device__ __forceinline__ int splits_of(const Args &A, int64_t W) {
    int s = A.tc_parts_for[0];
#pragma unroll
    for (int i = 1; i < kPlans; ++i)
        if (i < A.tc_plans && W >= A.tc_from[i]) s = A.tc_parts_for[i];
    return s;
}

// How many chunks W steps are cut into: chunk c of n is [W c / n, W (c + 1) / n), n <= W, so
// that none is empty and an item's chunks are consecutive.  One per SM while there is a
// step for each, more of them from four steps each on (32 sequences of 33 to 900 keys
// behind a prefix of 4096: 23.2 us; chunks of three steps 23.6, of six 23.4, as many chunks
// as fit 23.7, one per SM 27.6), and no more than fit beside the prefix kernel.
__device__ __forceinline__ int64_t chunk_count(const Args &A, int64_t W) {
    int64_t n = W / 4 > kSms ? W / 4 : kSms;
    if (n > A.grid) n = A.grid;
    if (A.tc_items) {
        const int64_t free = int64_t(kSms - A.tc_items * splits_of(A, W)) * A.resident;
        if (free > 0 && n > free) n = free;
    }
    return n < W ? n : W;
}
__device__ __forceinline__ int64_t chunk_start(int64_t c, int64_t W, int64_t n) { return n ? quot(W * c, n) : 0; }
__device__ __forceinline__ int64_t chunk_of(int64_t u, int64_t W, int64_t n) { return quot((u + 1) * n - 1, W); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 2^x is taken against this base: -inf (a row that has seen no key) must not
// meet itself.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

// Whether a score of a row, m, is so far from 0 that half a step of fp32 there is two powers of two of a weight and
// more: fma(s, scale2, -m), whose product is not rounded as m was, may then pass what 16 bits hold.
__device__ __forceinline__ bool far_score(float m) { return fabsf(m) >= 33554432.0f; }     // 2^25

// Four consecutive columns of a finished row.
template <typename T>
__device__ __forceinline__ void store_out(const trit_attn_job &J, int64_t at, float4 v) {
    if (J.out_dtype == TRIT_F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(J.out) + at) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<T *>(J.out) + at) =
            make_uint2(pack16<T>(v.x, v.y), pack16<T>(v.z, v.w));
}
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : m * 0.693147180559945309f + logf(l);
}

// trit_attn_prefix.cu: whether the prefix runs there, its layout, its launch.
bool prefix_on_tensor_cores(const trit_attn_job &J);
// most: the own steps if every length were the table's.  Sets the grid of the own-keys
// kernel too.
void prefix_layout(Args &A, int64_t most);
int64_t prefix_part_bytes(const Args &A);
cudaError_t launch_prefix(const Args &A, cudaStream_t s);

}  // namespace attn
}  // namespace trit
