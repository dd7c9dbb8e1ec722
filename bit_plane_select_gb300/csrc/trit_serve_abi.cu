// The extern "C" boundary of the decode step between the products, of prompts, of the
// 4-bit cache and of scoring: argument validation on the host, then dispatch.  Nothing is enqueued when it fails.
#include <math.h>

#include "trit_internal.cuh"

namespace trit {
namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxKeys = int64_t(1) << 30;    // prefix_len and table_pages * page_size
constexpr int kMaxHeads = 1024;
constexpr int64_t kMaxPromptRows = int64_t(1) << 27;

trit_status check_cache(const trit_kv_cache &c) {
    if (!c.k || !c.v || !aligned(c.k, 16) || !aligned(c.v, 16) || c.reserved != 0) return TRIT_E_ARG;
    if (c.dtype != TRIT_BF16 && c.dtype != TRIT_F16) return TRIT_E_ARG;
    if (c.page_stride < 0 || c.head_stride < 0 || c.slot_stride < 0 || c.page_stride % 8 ||
        c.head_stride % 8 || c.slot_stride % 8)
        return TRIT_E_ARG;
    if ((c.head_dim != 64 && c.head_dim != 128) || c.pages < 1 || c.heads < 1 || c.heads > kMaxHeads ||
        c.page_size < 1)
        return TRIT_E_SHAPE;
    return TRIT_OK;
}

trit_status check_cache4(const trit_kv4_cache &c) {
    if (!c.k || !c.v || !c.k_scale || !c.v_scale || !aligned(c.k, 16) || !aligned(c.v, 16) ||
        !aligned(c.k_scale, 16) || !aligned(c.v_scale, 16) || c.reserved != 0)
        return TRIT_E_ARG;
    if (c.page_stride < 0 || c.head_stride < 0 || c.slot_stride < 0) return TRIT_E_ARG;
    if ((c.head_dim != 64 && c.head_dim != 128) || c.pages < 1 || c.heads < 1 || c.heads > kMaxHeads ||
        c.page_size < 1)
        return TRIT_E_SHAPE;
    return TRIT_OK;
}

trit_status check_batch(const trit_kv_batch &b, int32_t page_size) {
    if (!b.table || !b.lens || !aligned(b.table, 4) || !aligned(b.lens, 4) || !aligned(b.new_lens, 4) ||
        !aligned(b.prefix_table, 4) || (b.prefix_len > 0 && !b.prefix_table))
        return TRIT_E_ARG;
    if (b.B < 1 || b.B > TRIT_MAX_SEQUENCES || b.T < 1 || b.T > (1 << 20) || b.table_pages < 1 ||
        b.table_stride < b.table_pages || b.prefix_len < 0 || b.prefix_len > kMaxKeys ||
        int64_t(b.table_pages) * page_size > kMaxKeys || b.prefix_pages < 0 ||
        int64_t(b.prefix_pages) * page_size < b.prefix_len)
        return TRIT_E_SHAPE;
    return TRIT_OK;
}

bool heads_ok(int32_t hq, int32_t heads) { return hq >= 1 && hq <= kMaxHeads && hq % heads == 0; }
bool half_type(int32_t t) { return t == TRIT_BF16 || t == TRIT_F16; }

// Rows and key steps of an attention over B sequences.
bool attn_rows_ok(const trit_kv_batch &b, int32_t page_size, int32_t q_heads) {
    return int64_t(b.B) * b.T * q_heads <= (int64_t(1) << 28) &&
           // steps of 64 keys are counted in 32 bits
           b.B * ((int64_t(b.table_pages) * page_size + 63) / 64) <= (int64_t(1) << 30);
}

// Everything of an attention job but its data pointers.
trit_status check_attn_sizes(const trit_attn_job &J) {
    trit_status st = check_cache(J.cache);
    if (st == TRIT_OK) st = check_batch(J.batch, J.cache.page_size);
    if (st != TRIT_OK) return st;
    if (J.flags != 0 || (J.out_dtype != TRIT_F32 && J.out_dtype != J.cache.dtype)) return TRIT_E_ARG;
    if (!heads_ok(J.q_heads, J.cache.heads) || !attn_rows_ok(J.batch, J.cache.page_size, J.q_heads)) return TRIT_E_SHAPE;
    return TRIT_OK;
}

trit_status check_attn4_sizes(const trit_attn4_job &J) {
    trit_status st = check_cache4(J.cache);
    if (st == TRIT_OK) st = check_batch(J.batch, J.cache.page_size);
    if (st != TRIT_OK) return st;
    if (J.flags != 0 || J.reserved != 0 || !half_type(J.dtype) || (J.out_dtype != TRIT_F32 && J.out_dtype != J.dtype))
        return TRIT_E_ARG;
    if (!heads_ok(J.q_heads, J.cache.heads) || !attn_rows_ok(J.batch, J.cache.page_size, J.q_heads)) return TRIT_E_SHAPE;
    return TRIT_OK;
}

bool err_ok(const uint32_t *err) { return err && aligned(err, 4); }

}  // namespace
}  // namespace trit

using namespace trit;

extern "C" {

TRIT_API trit_status trit_kv_append(const trit_kv_append_job *job, uint32_t *err_flag,
                                    trit_stream_t stream) {
    if (!job || !err_ok(err_flag)) return TRIT_E_ARG;
    const trit_kv_append_job &J = *job;
    trit_status st = check_cache(J.cache);
    if (st == TRIT_OK) st = check_batch(J.batch, J.cache.page_size);
    if (st != TRIT_OK) return st;
    if (!J.k || !J.v || (J.q == nullptr) != (J.q_out == nullptr) || !aligned(J.q, 16) || !aligned(J.k, 16) ||
        !aligned(J.v, 16) || !aligned(J.q_out, 16) || !aligned(J.cos, 16) || !aligned(J.sin, 16) ||
        !aligned(J.q_gain, 16) || !aligned(J.k_gain, 16) || (J.flags & ~TRIT_ROPE_PAIRS) != 0 || J.reserved != 0 ||
        (J.src_dtype != TRIT_F32 && J.src_dtype != J.cache.dtype) || (J.rot > 0 && (!J.cos || !J.sin)))
        return TRIT_E_ARG;
    const int64_t unit = J.src_dtype == TRIT_F32 ? 4 : 8;
    if (J.q_stride < 0 || J.k_stride < 0 || J.v_stride < 0 || J.q_stride % unit || J.k_stride % unit ||
        J.v_stride % unit)
        return TRIT_E_ARG;
    if (J.rot < 0 || J.rot > J.cache.head_dim || J.rot % 8 || J.max_pos < 0 || (J.q && !heads_ok(J.q_heads, J.cache.heads)))
        return TRIT_E_SHAPE;
    // a warp per token and five vectors: counted in 32 bits
    if (int64_t(J.batch.B) * J.batch.T > (int64_t(1) << 24) ||
        int64_t(J.batch.B) * J.batch.T * ((J.q ? J.q_heads : 0) + 2 * J.cache.heads) > (int64_t(1) << 31))
        return TRIT_E_SHAPE;
    if ((J.q_gain || J.k_gain) && (!isfinite(J.eps) || J.eps < 0.0f)) return TRIT_E_SCALE;
    st = abi_check_device();
    if (st != TRIT_OK) return st;
    const cudaError_t e = launch_kv_append(J, err_flag, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TRIT_OK : abi_cuda_fail(e);
}

TRIT_API int64_t trit_attn_workspace_bytes(const trit_attn_job *job) {
    return job && check_attn_sizes(*job) == TRIT_OK ? attn_workspace_bytes(*job) : -1;
}

TRIT_API trit_status trit_attn_paged(const trit_attn_job *job, uint32_t *err_flag,
                                     trit_stream_t stream) {
    if (!job || !err_ok(err_flag)) return TRIT_E_ARG;
    const trit_attn_job &J = *job;
    trit_status st = check_attn_sizes(J);
    if (st != TRIT_OK) return st;
    if (!J.q || !J.out || !J.workspace || !aligned(J.q, 16) || !aligned(J.out, 16) || !aligned(J.lse, 4) ||
        !aligned(J.workspace, 16) || J.q_stride < 0 || J.q_stride % 8)
        return TRIT_E_ARG;
    if (!isfinite(J.scale)) return TRIT_E_SCALE;
    if (J.workspace_bytes < attn_workspace_bytes(J)) return TRIT_E_SCRATCH;
    st = abi_check_device();
    if (st != TRIT_OK) return st;
    const cudaError_t e = launch_attn_paged(J, err_flag, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TRIT_OK : abi_cuda_fail(e);
}

TRIT_API trit_status trit_draft_verify(const trit_verify_job *job, uint32_t *err_flag,
                                       trit_stream_t stream) {
    if (!job || !err_ok(err_flag)) return TRIT_E_ARG;
    const trit_verify_job &J = *job;
    if (!J.p || !J.q || !J.draft || !J.u || !J.race || !J.tokens || !J.accepted || J.flags != 0)
        return TRIT_E_ARG;
    if (J.dtype != TRIT_F32 && J.dtype != TRIT_BF16 && J.dtype != TRIT_F16) return TRIT_E_ARG;
    const uintptr_t e = J.dtype == TRIT_F32 ? 4 : 2;
    if (!aligned(J.p, e) || !aligned(J.q, e) || !aligned(J.draft, 4) || !aligned(J.n_draft, 4) || !aligned(J.u, 4) ||
        !aligned(J.race, 4) || !aligned(J.tokens, 4) || !aligned(J.accepted, 4))
        return TRIT_E_ARG;
    if (J.p_seq_stride < 0 || J.p_tok_stride < 0 || J.q_seq_stride < 0 || J.q_tok_stride < 0 || J.race_stride < 0)
        return TRIT_E_ARG;
    if (J.B < 1 || J.B > 65535 || J.T < 1 || J.T > (1 << 20) || J.V < 1 || J.V > kMaxRows) return TRIT_E_SHAPE;
    const trit_status st = abi_check_device();
    if (st != TRIT_OK) return st;
    const cudaError_t ce = launch_draft_verify(J, err_flag, reinterpret_cast<cudaStream_t>(stream));
    return ce == cudaSuccess ? TRIT_OK : abi_cuda_fail(ce);
}

TRIT_API trit_status trit_kv4_append(const trit_kv4_append_job *job, uint32_t *err_flag,
                                     trit_stream_t stream) {
    if (!job || !err_ok(err_flag)) return TRIT_E_ARG;
    const trit_kv4_append_job &J = *job;
    trit_status st = check_cache4(J.cache);
    if (st == TRIT_OK) st = check_batch(J.batch, J.cache.page_size);
    if (st != TRIT_OK) return st;
    if (!J.k || !J.v || (J.q == nullptr) != (J.q_out == nullptr) || !aligned(J.q, 16) || !aligned(J.k, 16) ||
        !aligned(J.v, 16) || !aligned(J.q_out, 16) || !aligned(J.starts, 4) || !aligned(J.cos, 16) ||
        !aligned(J.sin, 16) || !aligned(J.q_gain, 16) || !aligned(J.k_gain, 16) || (J.flags & ~TRIT_ROPE_PAIRS) != 0 ||
        !half_type(J.dtype) || (J.src_dtype != TRIT_F32 && J.src_dtype != J.dtype) ||
        (J.rot > 0 && (!J.cos || !J.sin)) || (J.starts && J.batch.new_lens))
        return TRIT_E_ARG;
    const int64_t unit = J.src_dtype == TRIT_F32 ? 4 : 8;
    if (J.q_stride < 0 || J.k_stride < 0 || J.v_stride < 0 || J.q_stride % unit || J.k_stride % unit ||
        J.v_stride % unit)
        return TRIT_E_ARG;
    if (J.rot < 0 || J.rot > J.cache.head_dim || J.rot % 8 || J.max_pos < 0 || (J.q && !heads_ok(J.q_heads, J.cache.heads)))
        return TRIT_E_SHAPE;
    if (J.rows < 1 || J.rows > (int64_t(1) << 24) || (!J.starts && J.rows != int64_t(J.batch.B) * J.batch.T) ||
        J.rows * ((J.q ? J.q_heads : 0) + 2 * J.cache.heads) > (int64_t(1) << 31))
        return TRIT_E_SHAPE;
    if ((J.q_gain || J.k_gain) && (!isfinite(J.eps) || J.eps < 0.0f)) return TRIT_E_SCALE;
    st = abi_check_device();
    if (st != TRIT_OK) return st;
    const cudaError_t e = launch_kv4_append(J, err_flag, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TRIT_OK : abi_cuda_fail(e);
}

TRIT_API trit_status trit_kv4_read(const trit_kv4_read_job *job, uint32_t *err_flag,
                                   trit_stream_t stream) {
    if (!job || !err_ok(err_flag)) return TRIT_E_ARG;
    const trit_kv4_read_job &J = *job;
    trit_status st = check_cache4(J.cache);
    if (st == TRIT_OK) st = check_batch(J.batch, J.cache.page_size);
    if (st != TRIT_OK) return st;
    if (!J.k || !J.v || !J.starts || !aligned(J.k, 16) || !aligned(J.v, 16) || !aligned(J.starts, 4) ||
        !half_type(J.dtype) || J.flags != 0)
        return TRIT_E_ARG;
    if (J.rows < 1 || J.rows > kMaxPromptRows || J.rows * J.cache.heads > (int64_t(1) << 31)) return TRIT_E_SHAPE;
    st = abi_check_device();
    if (st != TRIT_OK) return st;
    const cudaError_t e = launch_kv4_read(J, err_flag, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TRIT_OK : abi_cuda_fail(e);
}

TRIT_API int64_t trit_attn4_workspace_bytes(const trit_attn4_job *job) {
    return job && check_attn4_sizes(*job) == TRIT_OK ? attn4_workspace_bytes(*job) : -1;
}

TRIT_API trit_status trit_attn_paged4(const trit_attn4_job *job, uint32_t *err_flag,
                                      trit_stream_t stream) {
    if (!job || !err_ok(err_flag)) return TRIT_E_ARG;
    const trit_attn4_job &J = *job;
    trit_status st = check_attn4_sizes(J);
    if (st != TRIT_OK) return st;
    if (!J.q || !J.out || !J.workspace || !aligned(J.q, 16) || !aligned(J.out, 16) || !aligned(J.lse, 4) ||
        !aligned(J.workspace, 16) || J.q_stride < 0 || J.q_stride % 8)
        return TRIT_E_ARG;
    if (!isfinite(J.scale)) return TRIT_E_SCALE;
    if (J.workspace_bytes < attn4_workspace_bytes(J)) return TRIT_E_SCRATCH;
    st = abi_check_device();
    if (st != TRIT_OK) return st;
    const cudaError_t e = launch_attn_paged4(J, err_flag, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TRIT_OK : abi_cuda_fail(e);
}

TRIT_API trit_status trit_attn_prompt(const trit_prompt_job *job, uint32_t *err_flag,
                                      trit_stream_t stream) {
    if (!job || !err_ok(err_flag)) return TRIT_E_ARG;
    const trit_prompt_job &J = *job;
    if (!J.q || !J.out || (J.k_rows > 0 && (!J.k || !J.v)) || !J.q_starts || !aligned(J.q, 16) || !aligned(J.k, 16) ||
        !aligned(J.v, 16) || !aligned(J.out, 16) || !aligned(J.lse, 4) || !aligned(J.q_starts, 4) ||
        !aligned(J.k_starts, 4) || !half_type(J.dtype) || (J.out_dtype != TRIT_F32 && J.out_dtype != J.dtype) || J.flags != 0)
        return TRIT_E_ARG;
    if ((J.head_dim != 64 && J.head_dim != 128) || J.heads < 1 || J.heads > kMaxHeads || !heads_ok(J.q_heads, J.heads) ||
        J.B < 1 || J.B > TRIT_MAX_SEQUENCES || J.q_rows < 1 || J.q_rows > kMaxPromptRows || J.k_rows < 0 ||
        J.k_rows > kMaxPromptRows || J.q_rows * J.q_heads > (int64_t(1) << 31))
        return TRIT_E_SHAPE;
    const int64_t q_row = int64_t(J.q_heads) * J.head_dim, k_row = int64_t(J.heads) * J.head_dim;
    const int64_t most = int64_t(1) << 38;      // what a copy's descriptor holds
    if (J.q_stride % 8 || J.k_stride % 8 || J.v_stride % 8 || J.q_stride < q_row || J.k_stride < k_row ||
        J.v_stride < k_row || J.q_stride >= most || J.k_stride >= most || J.v_stride >= most)
        return TRIT_E_ARG;
    if (!isfinite(J.scale) || !(J.scale > 0.0f)) return TRIT_E_SCALE;
    const trit_status st = abi_check_device();
    if (st != TRIT_OK) return st;
    const cudaError_t e = launch_attn_prompt(J, err_flag, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TRIT_OK : abi_cuda_fail(e);
}

TRIT_API trit_status trit_logprobs(const trit_logprob_job *job, uint32_t *err_flag,
                                   trit_stream_t stream) {
    if (!job || !err_ok(err_flag)) return TRIT_E_ARG;
    const trit_logprob_job &J = *job;
    if (!J.logits || (J.tokens == nullptr) != (J.logprob == nullptr) || (J.top_n > 0) != (J.top_tokens != nullptr) ||
        (J.top_n > 0) != (J.top_logprobs != nullptr) || J.flags != 0 || J.reserved != 0)
        return TRIT_E_ARG;
    if (J.dtype != TRIT_F32 && !half_type(J.dtype)) return TRIT_E_ARG;
    if (!aligned(J.logits, J.dtype == TRIT_F32 ? 4 : 2) || !aligned(J.tokens, 4) || !aligned(J.logprob, 4) ||
        !aligned(J.entropy, 4) || !aligned(J.top_tokens, 4) || !aligned(J.top_logprobs, 4) || J.stride < 0)
        return TRIT_E_ARG;
    if (J.rows < 1 || J.rows > (int64_t(1) << 24) || J.V < 1 || J.V > kMaxRows || J.top_n < 0 || J.top_n > TRIT_MAX_TOP)
        return TRIT_E_SHAPE;
    const trit_status st = abi_check_device();
    if (st != TRIT_OK) return st;
    const cudaError_t e = launch_logprobs(J, err_flag, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TRIT_OK : abi_cuda_fail(e);
}

}  // extern "C"
