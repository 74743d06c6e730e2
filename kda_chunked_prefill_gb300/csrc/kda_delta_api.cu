// Host side of kda_gated_delta_chunk_fwd and kda_gated_delta_decode_fwd: argument checks and launches.
#include <cuda_runtime.h>

#include "kda.h"
#include "kda_checks.h"
#include "kda_delta.h"

namespace {

using kda::checks::aligned;

// The checks both entry points share; fills p. KDA_OK: the call may proceed.
kda_status_t delta_args(const void *q, const void *k, const void *v, const float *g, const float *beta, int32_t num_seqs,
                        int64_t tokens, int32_t num_heads, int32_t num_qk_heads, int32_t dk, int32_t dv, int64_t qs,
                        int64_t ks, int64_t vs, const float *s0, float scale, void *o, float *sT, int32_t *status,
                        kda::delta::Params *p) {
    if (dk != KDA_HEAD_DIM || dv != KDA_HEAD_DIM) return KDA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || tokens < 0 || num_heads < 1 || num_qk_heads < 1 || num_heads % num_qk_heads != 0)
        return KDA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(num_seqs) * num_heads > 0x7fffffffLL / 4) return KDA_ERR_INVALID_ARG;
    if (tokens > (int64_t{1} << 40) / (static_cast<int64_t>(num_heads) * KDA_HEAD_DIM)) return KDA_ERR_INVALID_ARG;
    if (tokens > kda::checks::kMaxTokens) return KDA_ERR_UNSUPPORTED;
    if (!kda::checks::scale_ok(scale)) return KDA_ERR_INVALID_ARG;
    const int64_t qw = static_cast<int64_t>(num_qk_heads) * KDA_HEAD_DIM, vw = static_cast<int64_t>(num_heads) * KDA_HEAD_DIM;
    if (qs < qw || ks < qw || vs < vw || qs % 8 || ks % 8 || vs % 8) return KDA_ERR_INVALID_ARG;
    // a tensor map's strides are below 2^40 bytes, and so is the last token's offset
    if (tokens > 0 && (qs > (int64_t{1} << 38) / tokens || ks > (int64_t{1} << 38) / tokens || vs > (int64_t{1} << 38) / tokens))
        return KDA_ERR_UNSUPPORTED;
    if (num_seqs > 0 && tokens > 0) {
        if (!q || !k || !v || !g || !beta || !o) return KDA_ERR_INVALID_ARG;
        if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 4) || !aligned(beta, 4) || !aligned(o, 16))
            return KDA_ERR_INVALID_ARG;
    }
    if ((s0 && !aligned(s0, 16)) || (sT && !aligned(sT, 16)) || (status && !aligned(status, 4))) return KDA_ERR_INVALID_ARG;
    p->q = static_cast<const __nv_bfloat16 *>(q);
    p->k = static_cast<const __nv_bfloat16 *>(k);
    p->v = static_cast<const __nv_bfloat16 *>(v);
    p->qs = qs;
    p->ks = ks;
    p->vs = vs;
    p->g = g;
    p->beta = beta;
    p->cu = nullptr;
    p->steps = 0;
    p->N = num_seqs;
    p->T = tokens;
    p->longest = -1;
    p->listed = nullptr;
    p->list = nullptr;
    p->most = 0;
    p->H = num_heads;
    p->rep = num_heads / num_qk_heads;
    p->s0 = s0;
    p->scale = scale;
    p->o = static_cast<__nv_bfloat16 *>(o);
    p->sT = sT;
    p->status = status;
    return KDA_OK;
}

kda_status_t chunk_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta, const int32_t *cu_seqlens,
                       int32_t num_seqs, int64_t total_tokens, int32_t num_heads, int32_t num_qk_heads, int32_t head_dim_k,
                       int32_t head_dim_v, int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride,
                       const float *initial_state, float scale, void *o, float *final_state, int32_t *status_dev,
                       void *workspace, size_t workspace_bytes, kda_stream_t stream, int32_t withhold) {
    kda::delta::Params p;
    const kda_status_t rc = delta_args(q, k, v, g, beta, num_seqs, total_tokens, num_heads, num_qk_heads, head_dim_k,
                                       head_dim_v, q_token_stride, k_token_stride, v_token_stride, initial_state, scale,
                                       o, final_state, status_dev, &p);
    if (rc != KDA_OK) return rc;
    if (num_seqs > 0 && (!cu_seqlens || !aligned(cu_seqlens, 4))) return KDA_ERR_INVALID_ARG;
    const size_t need = kda_gated_delta_chunk_fwd_workspace_size(num_seqs, total_tokens, num_heads);
    if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (status_dev && cudaMemsetAsync(status_dev, 0, sizeof(int32_t), s) != cudaSuccess) return KDA_ERR_CUDA;
    if (num_seqs == 0) return KDA_OK;
    p.cu = cu_seqlens;
    return kda::delta::launch_chunked(p, workspace, s, withhold) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

extern "C" {

kda_status_t kda_gated_delta_chunk_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                       const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                       int32_t num_heads, int32_t num_qk_heads, int32_t head_dim_k, int32_t head_dim_v,
                                       int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride,
                                       const float *initial_state, float scale, void *o, float *final_state,
                                       int32_t *status_dev, void *workspace, size_t workspace_bytes,
                                       kda_stream_t stream) {
    return chunk_fwd(q, k, v, g, beta, cu_seqlens, num_seqs, total_tokens, num_heads, num_qk_heads, head_dim_k, head_dim_v,
                     q_token_stride, k_token_stride, v_token_stride, initial_state, scale, o, final_state, status_dev,
                     workspace, workspace_bytes, stream, -1);
}

kda_status_t kda_gated_delta_chunk_fwd_debug(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                             const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                             int32_t num_heads, int32_t num_qk_heads, int32_t head_dim_k,
                                             int32_t head_dim_v, int64_t q_token_stride, int64_t k_token_stride,
                                             int64_t v_token_stride, const float *initial_state, float scale, void *o,
                                             float *final_state, int32_t *status_dev, void *workspace,
                                             size_t workspace_bytes, kda_stream_t stream, int32_t withhold) {
    if (withhold < -1) return KDA_ERR_INVALID_ARG;
    return chunk_fwd(q, k, v, g, beta, cu_seqlens, num_seqs, total_tokens, num_heads, num_qk_heads, head_dim_k, head_dim_v,
                     q_token_stride, k_token_stride, v_token_stride, initial_state, scale, o, final_state, status_dev,
                     workspace, workspace_bytes, stream, withhold);
}

size_t kda_gated_delta_chunk_fwd_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t num_heads) {
    if (num_seqs < 1 || total_tokens < 1 || num_heads < 1) return 0;
    if (total_tokens > kda::checks::kMaxTokens || total_tokens > (int64_t{1} << 40) / num_heads) return 0;
    return kda::delta::chunked_workspace_bytes(num_seqs, total_tokens, num_heads);
}

kda_status_t kda_gated_delta_decode_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                        int32_t num_seqs, int32_t tokens_per_seq, int32_t num_heads,
                                        int32_t num_qk_heads, int32_t head_dim_k, int32_t head_dim_v,
                                        int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride,
                                        const float *initial_state, float scale, void *o, float *final_state,
                                        int32_t *status_dev, kda_stream_t stream) {
    if (tokens_per_seq < 0 || tokens_per_seq > KDA_DECODE_MAX_TOKENS) return KDA_ERR_INVALID_ARG;
    kda::delta::Params p;
    const kda_status_t rc =
        delta_args(q, k, v, g, beta, num_seqs, static_cast<int64_t>(num_seqs < 0 ? 0 : num_seqs) * tokens_per_seq, num_heads,
                   num_qk_heads, head_dim_k, head_dim_v, q_token_stride, k_token_stride, v_token_stride, initial_state,
                   scale, o, final_state, status_dev, &p);
    if (rc != KDA_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (status_dev && cudaMemsetAsync(status_dev, 0, sizeof(int32_t), s) != cudaSuccess) return KDA_ERR_CUDA;
    if (num_seqs == 0) return KDA_OK;
    p.steps = tokens_per_seq;
    return kda::delta::launch_recurrent(p, s) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
