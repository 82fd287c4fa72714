// C-ABI entry points of the attention-side calls: host-side argument checks and dispatch.
#include <cmath>
#include <cstdint>

#include "kv.cuh"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
ssd_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }
bool dtype_ok(int32_t d) { return d == SSD_F32 || d == SSD_BF16; }
int elem_bytes(int32_t d) { return d == SSD_BF16 ? 2 : 4; }

// strides in elements of rows of `row` elements, in whole 16-byte pieces
bool stride_ok(int64_t stride, int64_t row, int32_t dtype) {
    return stride >= row && stride <= (int64_t{1} << 40) && stride * elem_bytes(dtype) % 16 == 0;
}

// slots and block ids fit 32 bits, blocks do not overlap
bool pages_ok(int32_t block_size, int32_t num_blocks, int64_t block_stride, int64_t row, int32_t dtype) {
    return block_size >= 1 && num_blocks >= 1 && (int64_t)block_size * num_blocks < (int64_t{1} << 31) &&
           stride_ok(block_stride, (int64_t)block_size * row, dtype);
}

// the same of a cache in 8 bits, in pieces of 8 codes
bool pages8_ok(int32_t block_size, int32_t num_blocks, int64_t block_stride, int64_t row) {
    return block_size >= 1 && num_blocks >= 1 && (int64_t)block_size * num_blocks < (int64_t{1} << 31) &&
           block_stride >= (int64_t)block_size * row && block_stride <= (int64_t{1} << 40) && block_stride % 8 == 0;
}

// positions up to a key tile's end fit 32 bits
bool table_ok(int32_t table_cols, int32_t block_size) {
    return table_cols >= 0 && (int64_t)table_cols * block_size <= INT32_MAX - 1024;
}

bool heads_ok(int32_t H, int32_t G, int32_t D) {
    return H > 0 && G > 0 && H % G == 0 && H <= 65536 && D > 0 && D <= 256 && D % 8 == 0;
}

ssd_status_t check_tables(const kv_tables_args *a) {
    if (!a) return SSD_ERR_INVALID_ARG;
    if (a->num_reqs < 0 || a->max_tokens < 0 || a->block_size < 1 || a->table_cols < 0 || a->free_capacity < 0 ||
        a->num_blocks < 0 || (int64_t)a->block_size * a->num_blocks >= (int64_t{1} << 31))
        return SSD_ERR_INVALID_ARG;
    if (!a->ring_in || !a->ring_out || !a->cu_seqlens) return SSD_ERR_INVALID_ARG;
    if (a->num_reqs > 0 && (!a->context_lens || !a->new_lens || !a->reserved_lens || !a->seq_lens || !a->reserved_out))
        return SSD_ERR_INVALID_ARG;
    // every CTA reads the inputs again while others write outputs already
    const int32_t *const outs[] = {a->ring_out, a->cu_seqlens, a->seq_lens, a->reserved_out, a->slots, a->positions,
                                   a->token_req};
    const int32_t *const ins[] = {a->context_lens, a->new_lens, a->reserved_lens, a->ring_in, a->free_ring, a->block_table};
    for (const int32_t *o : outs)
        for (const int32_t *i : ins)
            if (o && o == i) return SSD_ERR_INVALID_ARG;
    if (a->num_reqs > 0 && a->table_cols > 0 && !a->block_table) return SSD_ERR_INVALID_ARG;
    if (a->free_capacity > 0 && !a->free_ring) return SSD_ERR_INVALID_ARG;
    if (a->max_tokens > 0 && (!a->slots || !a->positions)) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

ssd_status_t check_qk(const kv_qk_args *a) {
    if (!a) return SSD_ERR_INVALID_ARG;
    if (a->total_tokens < 0 || !heads_ok(a->nheads, a->kv_heads, a->headdim) || !dtype_ok(a->dtype))
        return SSD_ERR_INVALID_ARG;
    if (a->rotary_dim < 0 || a->rotary_dim > a->headdim || a->rotary_dim % 2 != 0 || a->max_position < 0)
        return SSD_ERR_INVALID_ARG;
    if (std::isnan(a->eps) || a->eps < 0.f) return SSD_ERR_INVALID_ARG;
    const int64_t row = (int64_t)a->kv_heads * a->headdim;
    if (!stride_ok(a->q_stride, (int64_t)a->nheads * a->headdim, a->dtype) || !stride_ok(a->k_stride, row, a->dtype))
        return SSD_ERR_INVALID_ARG;
    if (a->total_tokens == 0) return SSD_OK;
    if (!a->q || !a->k || !a->q_out || !aligned16(a->q) || !aligned16(a->k) || !aligned16(a->q_out) ||
        (a->k_out && !aligned16(a->k_out)))
        return SSD_ERR_INVALID_ARG;
    if (a->rotary_dim > 0 && (!a->cos_sin || !a->positions || !aligned4(a->positions))) return SSD_ERR_INVALID_ARG;
    // a row is only overwritten in place by the lanes that read it
    if ((a->q_out == a->q && a->q_stride != (int64_t)a->nheads * a->headdim) ||
        (a->k_out == a->k && a->k_stride != row))
        return SSD_ERR_INVALID_ARG;
    if ((a->k_cache == nullptr) != (a->v_cache == nullptr) || (a->k_cache == nullptr) != (a->slots == nullptr))
        return SSD_ERR_INVALID_ARG;
    if (a->k_cache) {
        if (!a->v || !aligned16(a->v) || !aligned16(a->k_cache) || !aligned16(a->v_cache) || !aligned4(a->slots) ||
            !stride_ok(a->v_stride, row, a->dtype) ||
            !pages_ok(a->block_size, a->num_blocks, a->cache_block_stride, row, a->dtype))
            return SSD_ERR_INVALID_ARG;
    }
    return SSD_OK;
}

ssd_status_t check_attention(const kv_attention_args *a, bool k8 = false) {
    if (!a) return SSD_ERR_INVALID_ARG;
    if (a->total_tokens < 0 || a->num_seqs < 0 || !heads_ok(a->nheads, a->kv_heads, a->headdim) || !dtype_ok(a->dtype))
        return SSD_ERR_INVALID_ARG;
    if (a->table_cols < 0 || a->max_new_tokens < 0 || a->mask_words < 0 || (a->tree_mask && a->mask_words == 0) ||
        a->wait_limit_cycles < 0 || !std::isfinite(a->scale))
        return SSD_ERR_INVALID_ARG;
    const int64_t row = (int64_t)a->kv_heads * a->headdim;
    if (!(k8 ? pages8_ok(a->block_size, a->num_blocks, a->cache_block_stride, row)
             : pages_ok(a->block_size, a->num_blocks, a->cache_block_stride, row, a->dtype)) ||
        !table_ok(a->table_cols, a->block_size))
        return SSD_ERR_INVALID_ARG;
    if (!stride_ok(a->q_stride, (int64_t)a->nheads * a->headdim, a->dtype) ||
        !stride_ok(a->k_stride, row, a->dtype) || !stride_ok(a->v_stride, row, a->dtype))
        return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

ssd_status_t check_attention_pointers(const kv_attention_args *a) {
    if (!a->q || !a->k_new || !a->v_new || !a->k_cache || !a->v_cache || !a->cu_seqlens || !a->context_lens || !a->out ||
        (a->table_cols > 0 && !a->block_table))
        return SSD_ERR_INVALID_ARG;
    if (!aligned16(a->q) || !aligned16(a->k_new) || !aligned16(a->v_new) || !aligned16(a->k_cache) ||
        !aligned16(a->v_cache) || !aligned16(a->out) || !aligned4(a->tree_mask) || !aligned4(a->block_table) ||
        !aligned4(a->lse))
        return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

// whether two stretches of memory have a byte in common
bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

// whether a call over a cache in 8 bits runs on the tensor cores: the sizes of the 16-bit one, blocks that TMA can step over
bool fp8_tc(const kv_attention_args *a) { return ssd::kv_attention_tc_supported(*a) && a->cache_block_stride % 16 == 0; }

bool empty(const kv_attention_args *a) { return a->total_tokens == 0 || a->num_seqs == 0; }

ssd_status_t check_commit(const kv_commit_args *a) {
    if (!a) return SSD_ERR_INVALID_ARG;
    if (a->total_tokens < 0 || a->num_seqs < 0 || a->kv_heads < 1 || a->headdim < 1 || a->kv_heads > 65536 ||
        a->headdim > 65536 || !dtype_ok(a->dtype) || a->max_path < 0)
        return SSD_ERR_INVALID_ARG;
    const int64_t row = (int64_t)a->kv_heads * a->headdim;
    if (row * elem_bytes(a->dtype) % 16 != 0 || row > (1 << 24) || !stride_ok(a->k_stride, row, a->dtype) ||
        !stride_ok(a->v_stride, row, a->dtype) ||
        !pages_ok(a->block_size, a->num_blocks, a->cache_block_stride, row, a->dtype))
        return SSD_ERR_INVALID_ARG;
    if ((a->path == nullptr) != (a->path_lens == nullptr) || (a->path && a->max_path == 0) ||
        (!a->path && a->max_path > 0 && a->num_seqs > 0) ||  // without requests there is nothing to point at
        (a->context_lens == nullptr) != (a->context_out == nullptr))
        return SSD_ERR_INVALID_ARG;
    if ((int64_t)a->num_seqs * a->max_path >= (int64_t{1} << 31)) return SSD_ERR_INVALID_ARG;
    if (a->num_seqs > 0 && (a->path || a->context_out) && !a->cu_seqlens) return SSD_ERR_INVALID_ARG;
    if (a->total_tokens == 0) return SSD_OK;
    if (!a->k_new || !a->v_new || !a->slots || !a->k_cache || !a->v_cache || !aligned16(a->k_new) ||
        !aligned16(a->v_new) || !aligned16(a->k_cache) || !aligned16(a->v_cache) || !aligned4(a->slots))
        return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

ssd_status_t check_commit_fp8(const kv_commit_fp8_args *a) {
    if (!a) return SSD_ERR_INVALID_ARG;
    if (a->total_tokens < 0 || a->num_seqs < 0 || !heads_ok(a->kv_heads, a->kv_heads, a->headdim) || a->kv_heads > 65535 ||
        !dtype_ok(a->dtype) || a->max_path < 0)
        return SSD_ERR_INVALID_ARG;
    const int64_t row = (int64_t)a->kv_heads * a->headdim;
    if (!stride_ok(a->k_stride, row, a->dtype) || !stride_ok(a->v_stride, row, a->dtype) ||
        !pages8_ok(a->block_size, a->num_blocks, a->cache_block_stride, row) || !table_ok(a->table_cols, a->block_size))
        return SSD_ERR_INVALID_ARG;
    if ((a->path == nullptr) != (a->path_lens == nullptr) || (a->path && a->max_path == 0) ||
        (!a->path && a->max_path > 0 && a->num_seqs > 0) ||
        (int64_t)a->num_seqs * (a->max_path + 2ll) >= (int64_t{1} << 30))
        return SSD_ERR_INVALID_ARG;
    if ((int64_t)a->block_size * a->headdim > INT32_MAX) return SSD_ERR_INVALID_ARG;  // pieces of a block are counted in 32 bits
    if (a->num_seqs > 0 && (!a->cu_seqlens || !a->context_lens)) return SSD_ERR_INVALID_ARG;
    if (!aligned4(a->cu_seqlens) || !aligned4(a->context_lens) || !aligned4(a->path) || !aligned4(a->path_lens) ||
        !aligned4(a->context_out) || !aligned4(a->err_word))
        return SSD_ERR_INVALID_ARG;
    // what one CTA writes, others read
    const int64_t list = 4ll * a->num_seqs;
    if (overlap(a->context_out, list, a->context_lens, list) || overlap(a->context_out, list, a->cu_seqlens, list + 4) ||
        overlap(a->context_out, list, a->path_lens, list) || overlap(a->context_out, list, a->path, list * a->max_path) ||
        overlap(a->context_out, list, a->block_table, list * a->table_cols))
        return SSD_ERR_INVALID_ARG;
    if (a->total_tokens == 0 || a->num_seqs == 0) return SSD_OK;
    if (!a->k_new || !a->v_new || !a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale ||
        (a->table_cols > 0 && !a->block_table) || !aligned16(a->k_new) || !aligned16(a->v_new) || !aligned16(a->k_cache) ||
        !aligned16(a->v_cache) || !aligned4(a->k_scale) || !aligned4(a->v_scale) || !aligned4(a->block_table))
        return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

ssd_status_t check_read_fp8(const kv_read_fp8_args *a) {
    if (!a) return SSD_ERR_INVALID_ARG;
    if (a->total_tokens < 0 || a->num_seqs < 0 || !heads_ok(a->kv_heads, a->kv_heads, a->headdim) || !dtype_ok(a->dtype))
        return SSD_ERR_INVALID_ARG;
    const int64_t row = (int64_t)a->kv_heads * a->headdim;
    if (!pages8_ok(a->block_size, a->num_blocks, a->cache_block_stride, row) || !table_ok(a->table_cols, a->block_size))
        return SSD_ERR_INVALID_ARG;
    if (a->num_seqs > 0 && !a->cu_seqlens) return SSD_ERR_INVALID_ARG;
    if (!aligned4(a->cu_seqlens) || !aligned4(a->starts) || !aligned4(a->err_word)) return SSD_ERR_INVALID_ARG;
    if (a->total_tokens == 0 || a->num_seqs == 0) return SSD_OK;
    if (!a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale || !a->k_out || !a->v_out ||
        (a->table_cols > 0 && !a->block_table) || !aligned16(a->k_cache) || !aligned16(a->v_cache) ||
        !aligned4(a->k_scale) || !aligned4(a->v_scale) || !aligned16(a->k_out) || !aligned16(a->v_out) ||
        !aligned4(a->block_table))
        return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

ssd_status_t check_verify(const kv_verify_args *a) {
    if (!a) return SSD_ERR_INVALID_ARG;
    if (a->total_tokens < 0 || a->num_seqs < 0 || a->vocab < 1 || a->vocab > (1 << 18) || !dtype_ok(a->dtype) ||
        a->max_path < 1 || a->target_stride < a->vocab || a->target_stride > (int64_t{1} << 31) ||
        (a->draft_probs && (a->draft_stride < a->vocab || a->draft_stride > (int64_t{1} << 31))))
        return SSD_ERR_INVALID_ARG;
    if (a->num_seqs == 0) return SSD_OK;
    if (!a->cu_seqlens || !a->path || !a->path_lens || !a->accepted || !a->next_tokens) return SSD_ERR_INVALID_ARG;
    if (!aligned4(a->cu_seqlens) || !aligned4(a->path) || !aligned4(a->path_lens) || !aligned4(a->accepted) ||
        !aligned4(a->next_tokens) || !aligned4(a->err_word))
        return SSD_ERR_INVALID_ARG;
    if (a->total_tokens == 0) return SSD_OK;
    const uintptr_t most = (uintptr_t)elem_bytes(a->dtype) - 1;
    if (!a->tokens || !a->uniform || !a->target_probs || (reinterpret_cast<uintptr_t>(a->target_probs) & most) ||
        (reinterpret_cast<uintptr_t>(a->draft_probs) & most) || !aligned4(a->tokens) || !aligned4(a->parents) ||
        !aligned4(a->uniform))
        return SSD_ERR_INVALID_ARG;
    // The CTAs of a request walk down its tree each for itself: what one writes, the others must not read.
    const int64_t list = 4ll * a->num_seqs, line = 4ll * a->total_tokens, last = a->total_tokens - 1;
    const void *const outs[4] = {a->path, a->path_lens, a->accepted, a->next_tokens};
    for (int i = 0; i < 4; ++i) {
        const int64_t bytes = i == 0 ? list * a->max_path : list;
        if (overlap(outs[i], bytes, a->cu_seqlens, list + 4) || overlap(outs[i], bytes, a->tokens, line) ||
            overlap(outs[i], bytes, a->parents, line) || overlap(outs[i], bytes, a->uniform, line) ||
            overlap(outs[i], bytes, a->target_probs, (last * a->target_stride + a->vocab) * elem_bytes(a->dtype)) ||
            overlap(outs[i], bytes, a->draft_probs, (last * a->draft_stride + a->vocab) * elem_bytes(a->dtype)))
            return SSD_ERR_INVALID_ARG;
    }
    return SSD_OK;
}

}  // namespace

extern "C" ssd_status_t kv_block_tables(const kv_tables_args *a, ssd_stream_t stream) {
    const ssd_status_t st = check_tables(a);
    if (st != SSD_OK) return st;
    return from_cuda(ssd::kv_tables_launch(*a, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" ssd_status_t kv_qk_norm_rope(const kv_qk_args *a, ssd_stream_t stream) {
    const ssd_status_t st = check_qk(a);
    if (st != SSD_OK || a->total_tokens == 0) return st;
    return from_cuda(ssd::kv_qk_launch(*a, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" size_t kv_tree_attention_workspace_size(const kv_attention_args *a) {
    if (check_attention(a) != SSD_OK || empty(a)) return 0;
    return ssd::kv_attention_tc_supported(*a) ? ssd::kv_attention_tc_workspace(*a)
                                              : ssd::kv_attention_simt_workspace(*a);
}

extern "C" ssd_status_t kv_tree_attention(const kv_attention_args *a, void *workspace, size_t workspace_bytes,
                                          ssd_stream_t stream) {
    ssd_status_t st = check_attention(a);
    if (st != SSD_OK || empty(a)) return st;
    st = check_attention_pointers(a);
    if (st != SSD_OK) return st;
    const bool tc = ssd::kv_attention_tc_supported(*a);
    const size_t need = tc ? ssd::kv_attention_tc_workspace(*a) : ssd::kv_attention_simt_workspace(*a);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return SSD_ERR_WORKSPACE;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(tc ? ssd::kv_attention_tc_launch(*a, workspace, cs)
                        : ssd::kv_attention_simt_launch(*a, nullptr, workspace, cs));
}

extern "C" ssd_status_t kv_commit_tokens(const kv_commit_args *a, ssd_stream_t stream) {
    const ssd_status_t st = check_commit(a);
    if (st != SSD_OK || (a->total_tokens == 0 && (a->num_seqs == 0 || !a->context_out))) return st;
    if (a->num_seqs == 0 && a->max_path > 0) return st;  // no paths
    return from_cuda(ssd::kv_commit_launch(*a, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" ssd_status_t kv_commit_tokens_fp8(const kv_commit_fp8_args *a, ssd_stream_t stream) {
    const ssd_status_t st = check_commit_fp8(a);
    if (st != SSD_OK || a->num_seqs == 0 || (a->total_tokens == 0 && !a->context_out)) return st;
    return from_cuda(ssd::kv_commit_fp8_launch(*a, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" ssd_status_t kv_read_tokens_fp8(const kv_read_fp8_args *a, ssd_stream_t stream) {
    const ssd_status_t st = check_read_fp8(a);
    if (st != SSD_OK || a->num_seqs == 0 || a->total_tokens == 0) return st;
    return from_cuda(ssd::kv_read_fp8_launch(*a, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" size_t kv_tree_attention_fp8_workspace_size(const kv_attention_args *a) {
    if (check_attention(a, true) != SSD_OK || empty(a)) return 0;
    return fp8_tc(a) ? ssd::kv_attention_fp8_tc_workspace(*a) : ssd::kv_attention_simt_workspace(*a);
}

extern "C" ssd_status_t kv_tree_attention_fp8(const kv_attention_args *a, const float *k_scale, const float *v_scale,
                                              void *workspace, size_t workspace_bytes, ssd_stream_t stream) {
    ssd_status_t st = check_attention(a, true);
    if (st != SSD_OK || empty(a)) return st;
    st = check_attention_pointers(a);
    if (st != SSD_OK) return st;
    if (!k_scale || !v_scale || !aligned4(k_scale) || !aligned4(v_scale) || !aligned4(a->cu_seqlens) ||
        !aligned4(a->context_lens) || !aligned4(a->err_word))
        return SSD_ERR_INVALID_ARG;
    const bool tc = fp8_tc(a);
    const size_t need = tc ? ssd::kv_attention_fp8_tc_workspace(*a) : ssd::kv_attention_simt_workspace(*a);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return SSD_ERR_WORKSPACE;
    const ssd::fp8::Scales scales = {k_scale, v_scale};
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(tc ? ssd::kv_attention_fp8_tc_launch(*a, scales, workspace, cs)
                        : ssd::kv_attention_simt_launch(*a, &scales, workspace, cs));
}

extern "C" ssd_status_t kv_verify_tokens(const kv_verify_args *a, ssd_stream_t stream) {
    const ssd_status_t st = check_verify(a);
    if (st != SSD_OK || a->num_seqs == 0) return st;
    return from_cuda(ssd::kv_verify_launch(*a, reinterpret_cast<cudaStream_t>(stream)));
}
