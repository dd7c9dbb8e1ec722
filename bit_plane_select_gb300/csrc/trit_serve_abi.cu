// The extern "C" boundary of the decode step between the products: argument
// validation on the host, then dispatch.  Nothing is enqueued when it fails.
#include <math.h>

#include "trit_internal.cuh"

namespace trit {
namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxKeys = int64_t(1) << 30;    // prefix_len and table_pages * page_size
constexpr int kMaxHeads = 1024;

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

trit_status check_batch(const trit_kv_batch &b, const trit_kv_cache &c) {
    if (!b.table || !b.lens || !aligned(b.table, 4) || !aligned(b.lens, 4) || !aligned(b.new_lens, 4) ||
        !aligned(b.prefix_table, 4) || (b.prefix_len > 0 && !b.prefix_table))
        return TRIT_E_ARG;
    if (b.B < 1 || b.B > TRIT_MAX_SEQUENCES || b.T < 1 || b.T > (1 << 20) || b.table_pages < 1 ||
        b.table_stride < b.table_pages || b.prefix_len < 0 || b.prefix_len > kMaxKeys ||
        int64_t(b.table_pages) * c.page_size > kMaxKeys || b.prefix_pages < 0 ||
        int64_t(b.prefix_pages) * c.page_size < b.prefix_len)
        return TRIT_E_SHAPE;
    return TRIT_OK;
}

bool heads_ok(int32_t hq, const trit_kv_cache &c) {
    return hq >= 1 && hq <= kMaxHeads && hq % c.heads == 0;
}

// Everything of an attention job but its data pointers.
trit_status check_attn_sizes(const trit_attn_job &J) {
    trit_status st = check_cache(J.cache);
    if (st == TRIT_OK) st = check_batch(J.batch, J.cache);
    if (st != TRIT_OK) return st;
    if (J.flags != 0 || (J.out_dtype != TRIT_F32 && J.out_dtype != J.cache.dtype)) return TRIT_E_ARG;
    if (!heads_ok(J.q_heads, J.cache) ||
        int64_t(J.batch.B) * J.batch.T * J.q_heads > (int64_t(1) << 28) ||
        J.batch.B * ((int64_t(J.batch.table_pages) * J.cache.page_size + 63) / 64) > (int64_t(1) << 30))
        return TRIT_E_SHAPE;   // the last: steps of 64 keys are counted in 32 bits
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
    if (st == TRIT_OK) st = check_batch(J.batch, J.cache);
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
    if (J.rot < 0 || J.rot > J.cache.head_dim || J.rot % 8 || J.max_pos < 0 || (J.q && !heads_ok(J.q_heads, J.cache)))
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

}  // extern "C"
