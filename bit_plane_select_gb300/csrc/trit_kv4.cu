// trit_kv4_append and trit_kv4_read: into and out of the cache held in 4 bits.
//
// Append: norm and rotation as trit_kv_append, then per 64 columns of a key or value
//     z = fp16(min), s = fp16((max - min) / 15), c = rint((x - z) (1/s)) in 0..15.
// Read: s c + z in fp32, rounded once.
//
// Both are streams: (Hq + 2 Hkv) D values in and 2 Hq D + 1.125 Hkv D bytes out per new token,
// 1.125 Hkv D bytes in and 4 Hkv D out per key read; bound by memory for many
// tokens and by the latency of dependent loads (starts, lengths, page id, table rows) for
// few.  A lane holds eight (append also: four) consecutive columns, so that a group's
// least and greatest value are three (four) shuffles away and its eight codes are one word.
// With an SM's share of a copy's rate at 24 bytes a clock there are two dozen warp
// instructions for a lane's eight fp32 values, less than a group's range and codes take: so
// ranges come of three-input minima, values are held to fp16's range only where one is out of
// it, codes are rounded and packed by their fp32 bits, and codes are read where they stand in a word.
// Measured: 21,000 tokens of 20 + 2 x 5 heads of 128 fp32 columns appended and read back as bf16:
// 107 us, 5.0 TB/s (with conversions to whole numbers and back 114 us; loads of 32 bytes a lane no
// different); 366 tokens of 24 + 2 x 8 heads of 64 columns: 12.9 us, two launches and their latencies.
#include "trit_serve.cuh"

namespace trit {
namespace {

constexpr int kThreads = 128;
// of append, an SM: 80 registers, 24 warps, for which the forms of eight columns a lane spill 4 to 56 bytes a thread (five,
// which spill nothing: 111 us where six take 107)
constexpr int kCtas = 6;
constexpr int kGroup = TRIT_KV4_GROUP;
constexpr float kMost = 65504.0f;        // fp16's largest: values saturate there

struct Append4Args {
    trit_kv4_append_job J;
    uint32_t *err;
    int32_t chunks;      // warps per token
    int32_t page_shift;  // log2(page_size), or -1
};
// Warp steps of a warp, all in flight together.
constexpr int kSteps = 5;

// Whether sequence b's starts are in order, within [0, rows].
__device__ __forceinline__ bool starts_ok(const int32_t *starts, int b, int64_t rows) {
    return starts[b] >= 0 && starts[b + 1] >= starts[b] && starts[b + 1] <= rows;
}

// Of three, NaN if one is.
__device__ __forceinline__ float least(float a, float b, float c) {
    float d;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float greatest(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <typename T, typename S, int D, bool PAIRS, int W>
__global__ void __launch_bounds__(kThreads, kCtas) append4_kernel(const __grid_constant__ Append4Args A) {
    const trit_kv4_append_job &J = A.J;
    static_assert(W == 8 || (W == 4 && !PAIRS), "angles are read four at a time");
    constexpr int L = D / W;             // lanes of one head vector
    constexpr int V = 32 / L;            // vectors of a warp step
    constexpr int GL = kGroup / W;       // lanes of one group
    const int lane = threadIdx.x & 31, sub = lane % L, which = lane / L;
    const int64_t warp = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t row = warp / A.chunks;
    pdl_wait();
    pdl_launch();
    if (J.starts && blockIdx.x == 0)
        for (int i = threadIdx.x; i < J.batch.B; i += kThreads)
            if (!starts_ok(J.starts, i, J.rows) || J.starts[i + 1] - J.starts[i] > J.batch.T) raise_flag(A.err, TRIT_ERR_INDEX);
    if (row >= J.rows) return;
    const int first = int(warp - row * A.chunks) * kSteps;
    const int Hq = J.q ? J.q_heads : 0, Hkv = J.cache.heads, all = Hq + 2 * Hkv;
    const int j0 = sub * W, half = J.rot / 2;

    // every value first: the rest of the token's loads depend on one another
    const S *qp = static_cast<const S *>(J.q) + row * J.q_stride + j0;
    const S *kp = static_cast<const S *>(J.k) + row * J.k_stride + j0 - Hq * D;
    const S *vp = static_cast<const S *>(J.v) + row * J.v_stride + j0 - (Hq + Hkv) * D;
    float x[kSteps][W];
#pragma unroll
    for (int g = 0; g < kSteps; ++g) {
        int h = (first + g) * V + which;                    // vector of the token: q, k, v heads in turn
        h = h < all ? h : all - 1;
        load_row<W>((h < Hq ? qp : h < Hq + Hkv ? kp : vp) + h * D, x[g]);
    }

    // the token: of sequence b, the t-th of n
    int b, t, n;
    bool flag = false;
    if (J.starts) {
        b = sequence_of(J.starts, J.batch.B, row, lane);
        if (b < 0 || row >= J.starts[b + 1]) return;        // a row of no sequence
        t = int(row - J.starts[b]);
        n = J.starts[b + 1] - J.starts[b];
        n = n < J.batch.T ? n : J.batch.T;
    } else {
        b = int(row / J.batch.T);
        t = int(row - int64_t(b) * J.batch.T);
        const int given = J.batch.new_lens ? J.batch.new_lens[b] : J.batch.T;
        n = given < 0 ? 0 : given < J.batch.T ? given : J.batch.T;
        flag = n != given;
    }
    const int len = J.batch.lens[b];
    const int64_t own = int64_t(len) - n + t;
    const int64_t pos = J.batch.prefix_len + own;
    bool ok = t < n;
    int64_t slot_at = 0;
    const bool turns = j0 < J.rot;
    constexpr int CW = PAIRS ? W / 2 : W;
    float c[CW], s[CW];
#pragma unroll
    for (int i = 0; i < CW; ++i) {
        c[i] = 1.0f;
        s[i] = 0.0f;
    }
    if (ok) {
        const bool in = own >= 0 && (J.rot == 0 || pos < J.max_pos);
        // the lane's angles, and the page beside them
        if (in && turns) {
            const int64_t at = pos * half + (PAIRS ? j0 / 2 : j0 < half ? j0 : j0 - half);
            load_row<CW>(J.cos + at, c);
            load_row<CW>(J.sin + at, s);
        }
        const int64_t col = own < 0 ? -1 : A.page_shift >= 0 ? own >> A.page_shift : own / J.cache.page_size;
        int page = -1;
        if (in && col < J.batch.table_pages) page = J.batch.table[b * J.batch.table_stride + col];
        ok = page >= 0 && page < J.cache.pages;
        flag = flag || !ok;
        slot_at = page * J.cache.page_stride + (own - col * J.cache.page_size) * J.cache.slot_stride;
    }
    // the lane holding the rotation partners, and the sign of their sine (rot / 2 is a
    // multiple of W here)
    const int partner = !turns ? lane : (j0 < half ? lane + half / W : lane - half / W);
    if (!PAIRS && j0 < half) {
#pragma unroll
        for (int i = 0; i < CW; ++i) s[i] = -s[i];
    }
    T *q_out = static_cast<T *>(J.q_out) + row * Hq * D + j0;

#pragma unroll
    for (int g = 0; g < kSteps; ++g) {
        const int h = (first + g) * V + which;
        const bool is_q = h < Hq, is_v = h >= Hq + Hkv;
        float(&v)[W] = x[g];
        if (J.q_gain || J.k_gain) {                         // uniform: every lane shuffles
            float sum = v[0] * v[0];
#pragma unroll
            for (int i = 1; i < W; ++i) sum = fmaf(v[i], v[i], sum);
#pragma unroll
            for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            const float *gain = is_q ? J.q_gain : is_v ? nullptr : J.k_gain;
            if (gain) {
                const float r = rsqrtf(sum * (1.0f / D) + J.eps);
                float gg[W];
                load_row<W>(gain + j0, gg);
#pragma unroll
                for (int i = 0; i < W; ++i) v[i] = v[i] * r * gg[i];
            }
        }
        // the rotation, every operation rounded (no contraction): a key's codes follow from its values
        if (PAIRS) {
            if (turns && !is_v) {
#pragma unroll
                for (int i = 0; i < W / 2; ++i) {
                    const float a0 = v[2 * i], a1 = v[2 * i + 1], ci = c[i % CW], si = s[i % CW];
                    v[2 * i] = __fsub_rn(__fmul_rn(a0, ci), __fmul_rn(a1, si));
                    v[2 * i + 1] = __fadd_rn(__fmul_rn(a1, ci), __fmul_rn(a0, si));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float o = __shfl_sync(~0u, v[i], partner);
                if (turns && !is_v) v[i] = __fadd_rn(__fmul_rn(v[i], c[i % CW]), __fmul_rn(o, s[i % CW]));
            }
        }
        if ((first + g) * V + V - 1 < Hq) {                 // queries only: nothing to quantise
            if (!ok) {
#pragma unroll
                for (int i = 0; i < W; ++i) v[i] = 0.0f;
            }
            store_row<W>(q_out + h * D, v);
            continue;
        }
        if (is_q) {
            float y[W];
#pragma unroll
            for (int i = 0; i < W; ++i) y[i] = ok ? v[i] : 0.0f;
            store_row<W>(q_out + h * D, y);
        }
        // the group's range: every lane shuffles.  (NaN where a value is)
        float low = v[0], high = v[0];
#pragma unroll
        for (int i = 1; i + 1 < W; i += 2) {
            low = least(low, v[i], v[i + 1]);
            high = greatest(high, v[i], v[i + 1]);
        }
        low = least(low, low, v[W - 1]);
        high = greatest(high, high, v[W - 1]);
#pragma unroll
        for (int o = GL / 2; o; o >>= 1) {
            low = least(low, low, __shfl_xor_sync(~0u, low, o));
            high = greatest(high, high, __shfl_xor_sync(~0u, high, o));
        }
        const bool bad = !(low > -INFINITY && high < INFINITY);
        if (!(low >= -kMost && high <= kMost)) {
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = fminf(fmaxf(v[i], -kMost), kMost);
            low = fminf(fmaxf(low, -kMost), kMost);
            high = fminf(fmaxf(high, -kMost), kMost);
        }
        const __half sh = __float2half_rn(bad ? 0.0f : __fdiv_rn(__fsub_rn(high, low), 15.0f));
        const __half zh = __float2half_rn(bad ? __int_as_float(0x7fffffff) : low);
        const float sf = __half2float(sh), zf = __half2float(zh);
        const float inv = sf > 0.0f ? __fdiv_rn(1.0f, sf) : 0.0f;
        // 1.5 2^23 + c, rounded as rint, is 0x4b400000 + c in bits: a word of codes is their sum by 16^i, less
        // what the first parts add up to
        uint32_t word = 0;
#pragma unroll
        for (int i = W - 1; i >= 0; --i) {
            const float u = __fmul_rn(__fsub_rn(v[i], zf), inv);       // NaN only where the group is: code 0
            word = word * 16 + __float_as_uint(__fadd_rn(fminf(fmaxf(u, 0.0f), 15.0f), 12582912.0f));
        }
        word -= 0x4b400000u * 0x11111111u;                             // (of four codes' words the upper half is not used)
        if (is_q || h >= all || !ok) continue;
        const int64_t vec = slot_at + (is_v ? h - Hq - Hkv : h - Hq) * J.cache.head_stride;
        uint8_t *codes = (is_v ? J.cache.v : J.cache.k) + vec * (D / 2) + j0 / 2;
        if (W == 8) *reinterpret_cast<uint32_t *>(codes) = word;
        else *reinterpret_cast<uint16_t *>(codes) = uint16_t(word);
        if ((lane & (GL - 1)) == 0)
            static_cast<__half2 *>(is_v ? J.cache.v_scale : J.cache.k_scale)[vec * (D / kGroup) + j0 / kGroup] =
                __halves2half2(sh, zh);
    }
    if (flag) raise_flag(A.err, TRIT_ERR_INDEX);
}

template <typename T, typename S, int D>
cudaError_t launch_append_d(const Append4Args &A, int W, int64_t blocks, cudaStream_t s) {
    const dim3 grid{unsigned(blocks)}, block{kThreads};
    if (A.J.flags & TRIT_ROPE_PAIRS) return launch_pdl(append4_kernel<T, S, D, true, 8>, grid, block, 0, s, A);
    return W == 8 ? launch_pdl(append4_kernel<T, S, D, false, 8>, grid, block, 0, s, A)
                  : launch_pdl(append4_kernel<T, S, D, false, 4>, grid, block, 0, s, A);
}
template <typename T, typename S>
cudaError_t launch_append_s(const Append4Args &A, int W, int64_t blocks, cudaStream_t s) {
    return A.J.cache.head_dim == 128 ? launch_append_d<T, S, 128>(A, W, blocks, s)
                                     : launch_append_d<T, S, 64>(A, W, blocks, s);
}

int shift_of(int page_size) {
    for (int i = 0; i < 31; ++i)
        if (page_size == (1 << i)) return i;
    return -1;
}

struct Read4Args {
    trit_kv4_read_job J;
    uint32_t *err;
    int32_t chunks;      // warps per key
    int32_t page_shift;  // log2(page_size), or -1
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read4_kernel(const __grid_constant__ Read4Args A) {
    const trit_kv4_read_job &J = A.J;
    constexpr int W = 8, L = D / W, V = 32 / L;
    const int lane = threadIdx.x & 31, sub = lane % L, which = lane / L;
    const int64_t warp = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t row = warp / A.chunks;
    pdl_wait();
    pdl_launch();
    const int64_t P = J.batch.prefix_len, cap = int64_t(J.batch.table_pages) * J.cache.page_size;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < J.batch.B; i += kThreads) {
            const int64_t len = J.batch.lens[i];
            if (!starts_ok(J.starts, i, J.rows) || len < 0 || len > cap ||
                int64_t(J.starts[i + 1]) - J.starts[i] < P + len)
                raise_flag(A.err, TRIT_ERR_INDEX);
        }
    if (row >= J.rows) return;
    const int b = sequence_of(J.starts, J.batch.B, row, lane);
    if (b < 0 || row >= J.starts[b + 1]) return;
    int64_t len = J.batch.lens[b];
    len = len < 0 ? 0 : len < cap ? len : cap;
    const int64_t i = row - J.starts[b];
    if (i >= P + len) return;
    const int64_t key = i < P ? i : i - P;
    const int64_t col = A.page_shift >= 0 ? key >> A.page_shift : key / J.cache.page_size;
    const int page = i < P ? J.batch.prefix_table[col] : J.batch.table[b * J.batch.table_stride + col];
    const bool ok = page >= 0 && page < J.cache.pages;
    if (!ok) raise_flag(A.err, TRIT_ERR_INDEX);
    const int64_t slot_at = page * J.cache.page_stride + (key - col * J.cache.page_size) * J.cache.slot_stride;
    const int Hkv = J.cache.heads, first = int(warp - row * A.chunks) * kSteps;

    // vectors of the key: k, v heads in turn.  Their bytes: of codes D / 2, of pairs an eighth of that
    const int64_t step = J.cache.head_stride * (D / 2), at = slot_at * (D / 2) + sub * 4;
    const int64_t pair_at = slot_at * (D / 16) + sub * W / kGroup * 4;
    const uint8_t *const kc = J.cache.k + at, *const vc = J.cache.v + at - Hkv * step;
    const uint8_t *const ks = static_cast<const uint8_t *>(J.cache.k_scale) + pair_at;
    const uint8_t *const vs = static_cast<const uint8_t *>(J.cache.v_scale) + pair_at - Hkv * (step / 8);
    T *const k_out = static_cast<T *>(J.k) + row * Hkv * D + sub * W;
    T *const v_out = static_cast<T *>(J.v) + (row - 1) * Hkv * D + sub * W;
    const int h0 = first * V + which;
    int64_t off = h0 * step;
    uint32_t word[kSteps];
    __half2 sz[kSteps];
#pragma unroll
    for (int g = 0; g < kSteps; ++g) {
        const int h = h0 + g * V;
        word[g] = 0;
        sz[g] = __half2{};
        if (h < 2 * Hkv && ok) {
            const bool is_v = h >= Hkv;
            word[g] = __ldg(reinterpret_cast<const uint32_t *>((is_v ? vc : kc) + off));
            sz[g] = __ldg(reinterpret_cast<const __half2 *>((is_v ? vs : ks) + (off >> 3)));
        }
        off += V * step;
    }
#pragma unroll
    for (int g = 0; g < kSteps; ++g) {
        const int h = h0 + g * V;
        if (h >= 2 * Hkv) continue;
        const float2 f = __half22float2(sz[g]);
        // s, s / 16, s / 256, s / 4096 (exact) for the codes where they stand
        const float s[4] = {f.x, f.x * 0.0625f, f.x * 0.00390625f, f.x * 0.000244140625f};
        float y[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            // 2^23 + c 16^i, exactly, by its bits
            const float c = __uint_as_float(0x4b000000u | ((i < 4 ? word[g] : word[g] >> 16) & (15u << (4 * (i & 3))))) - 8388608.0f;
            y[i] = fmaf(c, s[i & 3], f.y);
        }
        store_row<W>((h >= Hkv ? v_out : k_out) + int64_t(h) * D, y);
    }
}

template <typename T>
cudaError_t launch_read(const Read4Args &A, int64_t blocks, cudaStream_t s) {
    const dim3 grid{unsigned(blocks)}, block{kThreads};
    return A.J.cache.head_dim == 128 ? launch_pdl(read4_kernel<T, 128>, grid, block, 0, s, A)
                                     : launch_pdl(read4_kernel<T, 64>, grid, block, 0, s, A);
}

}  // namespace

cudaError_t launch_kv4_append(const trit_kv4_append_job &J, uint32_t *err, cudaStream_t s) {
    Append4Args A;
    A.J = J;
    A.err = err;
    const int vectors = (J.q ? J.q_heads : 0) + 2 * J.cache.heads;
    // eight columns a lane, except where halves of the rotation do not start on eight
    const int W = (J.flags & TRIT_ROPE_PAIRS) || J.rot % 16 == 0 ? 8 : 4;
    const int per_step = 32 * W / J.cache.head_dim;
    const int steps = (vectors + per_step - 1) / per_step;
    A.chunks = (steps + kSteps - 1) / kSteps;
    A.page_shift = shift_of(J.cache.page_size);
    const int64_t warps = J.rows * A.chunks;
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (J.dtype == TRIT_BF16)
        return J.src_dtype == TRIT_F32 ? launch_append_s<__nv_bfloat16, float>(A, W, blocks, s)
                                       : launch_append_s<__nv_bfloat16, __nv_bfloat16>(A, W, blocks, s);
    return J.src_dtype == TRIT_F32 ? launch_append_s<__half, float>(A, W, blocks, s)
                                   : launch_append_s<__half, __half>(A, W, blocks, s);
}

cudaError_t launch_kv4_read(const trit_kv4_read_job &J, uint32_t *err, cudaStream_t s) {
    Read4Args A;
    A.J = J;
    A.err = err;
    const int per_step = 32 * 8 / J.cache.head_dim;
    const int steps = (2 * J.cache.heads + per_step - 1) / per_step;
    A.chunks = (steps + kSteps - 1) / kSteps;
    A.page_shift = shift_of(J.cache.page_size);
    const int64_t warps = J.rows * A.chunks;
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    return J.dtype == TRIT_BF16 ? launch_read<__nv_bfloat16>(A, blocks, s) : launch_read<__half>(A, blocks, s);
}

}  // namespace trit
