// latent_api.cu -- the latent-attention entry points of include/psw.h:
// argument checks (every error is returned before anything is launched) and
// dispatch to the launchers of latent_cache.cu, latent_decode.cu,
// latent_expand.cu and latent_prefill.cu.
#include <math.h>

#include "psw_internal.h"

using namespace psw;

namespace {

bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

int check_latent(const psw_latent_t* layer, LatentArgs* out) {
  if (layer == nullptr) return PSW_ENULL;
  if (layer->n_heads < 1 || layer->n_heads > 128) return PSW_EINVAL_HEADS;
  if ((layer->latent_dim != 256 && layer->latent_dim != 512) ||
      layer->rope_dim != kLatentRope || layer->nope_dim != kLatentNope ||
      layer->v_dim != kLatentV)
    return PSW_EINVAL_HDIM;
  if (!(layer->softcap >= 0.f) || !isfinite(layer->softcap)) return PSW_EINVAL_SOFTCAP;
  if (layer->window < 0) return PSW_EINVAL_WINDOW;
  if (layer->block_size != kBlockSize) return PSW_EINVAL_BLOCKSIZE;
  if (!(layer->scale > 0.f) || !isfinite(layer->scale)) return PSW_EINVAL_SCALE;
  out->n_heads = layer->n_heads;
  out->latent = layer->latent_dim;
  out->window = layer->window;
  // (beyond these fp32 cannot tell a cap from none, or from one that leaves every score 0)
  out->softcap = layer->softcap == 0.f ? 0.f : fminf(fmaxf(layer->softcap, 0x1p-100f), 0x1p100f);
  out->scale = layer->scale;
  return PSW_OK;
}

LatentPages pages_of(const psw_pages_t* pages, const void* pool, const float* row_scale) {
  return LatentPages{pool, row_scale, pages->block_table, pages->max_blocks_per_seq,
                     pages->num_blocks};
}

int ready(DeviceInfo* info, int32_t** err) {
  if (device_info(info) != cudaSuccess || info->cc_major != 10 || info->cc_minor != 3)
    return PSW_EDEVICE;
  *err = device_error_word();
  return PSW_OK;
}

bool row_stride_ok(int64_t s, int64_t least) { return s >= least && s % 8 == 0; }

int write_rows(const psw_latent_t* layer, const psw_latent_norm_t* norm, const void* ckv,
               int64_t ckv_stride, const void* q_rope, int64_t q_token_stride,
               int64_t q_head_stride, const int32_t* cu_new, const int32_t* past_lens,
               int32_t n_seqs, int32_t n_new_total, const psw_pages_t* pages, void* q_rope_out,
               int64_t qo_token_stride, int64_t qo_head_stride, void* pool, float* row_scale,
               psw_stream_t stream) {
  LatentArgs L;
  int rc = check_latent(layer, &L);
  if (rc != PSW_OK) return rc;
  if (norm == nullptr || ckv == nullptr || cu_new == nullptr || past_lens == nullptr ||
      pool == nullptr || (q_rope == nullptr) != (q_rope_out == nullptr))
    return PSW_ENULL;
  // (a base below 1 has frequencies above 1, whose angles the reduction does not cover)
  if (!(norm->theta >= 1.f) || !isfinite(norm->theta) || !(norm->eps >= 0.f) ||
      !isfinite(norm->eps))
    return PSW_EINVAL_ROPE;
  if ((rc = check_pages(pages)) != PSW_OK) return rc;
  if (n_seqs < 0) return PSW_EINVAL_NSEQS;
  if (n_new_total < 0) return PSW_ECAPACITY;
  if (!row_stride_ok(ckv_stride, L.row())) return PSW_EINVAL_STRIDE;
  if (q_rope != nullptr) {
    if (!row_stride_ok(q_token_stride, kLatentRope) ||
        !row_stride_ok(qo_token_stride, kLatentRope) ||
        !row_stride_ok(q_head_stride, kLatentRope) || !row_stride_ok(qo_head_stride, kLatentRope))
      return PSW_EINVAL_STRIDE;
    // in place means the same rows: another layout over them would be read
    // by one warp while a second one writes
    if (q_rope == q_rope_out &&
        (q_token_stride != qo_token_stride || q_head_stride != qo_head_stride))
      return PSW_EINVAL_STRIDE;
  }
  if (!aligned(ckv, 16) || !aligned(q_rope, 16) || !aligned(q_rope_out, 16) ||
      !aligned(pool, 16) || !aligned(norm->latent_weight, 16) || !aligned(row_scale, 16))
    return PSW_EALIGN;
  if (n_seqs == 0 || n_new_total == 0) return PSW_OK;
  DeviceInfo info;
  int32_t* err;
  if ((rc = ready(&info, &err)) != PSW_OK) return rc;
  const LatentRows q{q_rope, q_token_stride, q_head_stride,
                     q_rope_out, qo_token_stride, qo_head_stride};
  return launch_latent_write(L, norm->theta, norm->eps, norm->latent_weight, ckv, ckv_stride, q,
                             cu_new, past_lens, n_seqs, n_new_total,
                             pages_of(pages, pool, row_scale), pool,
                             row_scale, info.num_sms, err, reinterpret_cast<cudaStream_t>(stream));
}

int decode(const psw_latent_t* layer, const void* q, const void* pool, const float* row_scale,
           const psw_pages_t* pages, const int32_t* seq_lens, int32_t n_seqs, void* out,
           float* lse, void* ws, size_t ws_bytes, psw_stream_t stream) {
  LatentArgs L;
  int rc = check_latent(layer, &L);
  if (rc != PSW_OK) return rc;
  if (q == nullptr || pool == nullptr || seq_lens == nullptr || out == nullptr) return PSW_ENULL;
  if ((rc = check_pages(pages)) != PSW_OK) return rc;
  if (n_seqs < 0) return PSW_EINVAL_NSEQS;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(row_scale, 16) || !aligned(ws, 16))
    return PSW_EALIGN;
  if (static_cast<int64_t>(n_seqs) * (pages->max_blocks_per_seq + 12) * ((L.n_heads + 15) / 16) >
      INT32_MAX)
    return PSW_ECAPACITY;
  if (n_seqs == 0) return PSW_OK;
  if (ws == nullptr || ws_bytes < latent_decode_workspace(L, n_seqs)) return PSW_EWORKSPACE;
  DeviceInfo info;
  int32_t* err;
  if ((rc = ready(&info, &err)) != PSW_OK) return rc;
  return launch_latent_decode(L, q, pages_of(pages, pool, row_scale), seq_lens, n_seqs, out, lse,
                              ws, info.num_sms, err, reinterpret_cast<cudaStream_t>(stream));
}

int expand(const psw_latent_t* layer, const void* pool, const float* row_scale,
           const psw_pages_t* pages, const int32_t* cu_k, const int32_t* k_first, int32_t n_seqs,
           int32_t n_k_total, const void* w, void* kv, void* k_rope, psw_stream_t stream) {
  LatentArgs L;
  int rc = check_latent(layer, &L);
  if (rc != PSW_OK) return rc;
  if (pool == nullptr || cu_k == nullptr || w == nullptr || kv == nullptr || k_rope == nullptr)
    return PSW_ENULL;
  if ((rc = check_pages(pages)) != PSW_OK) return rc;
  if (n_seqs < 0) return PSW_EINVAL_NSEQS;
  if (n_k_total < 0) return PSW_ECAPACITY;
  if (!aligned(pool, 16) || !aligned(w, 16) || !aligned(kv, 16) || !aligned(k_rope, 16) ||
      !aligned(row_scale, 16))
    return PSW_EALIGN;
  if (n_seqs == 0 || n_k_total == 0) return PSW_OK;
  DeviceInfo info;
  int32_t* err;
  if ((rc = ready(&info, &err)) != PSW_OK) return rc;
  return launch_latent_expand(L, pages_of(pages, pool, row_scale), cu_k, k_first, n_seqs,
                              n_k_total, w, kv, k_rope, info.num_sms, err,
                              reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int psw_latent_workspace_bytes(const psw_latent_t* layer, int32_t n_seqs, size_t* bytes) {
  LatentArgs L;
  const int rc = check_latent(layer, &L);
  if (rc != PSW_OK) return rc;
  if (bytes == nullptr) return PSW_ENULL;
  if (n_seqs < 0) return PSW_EINVAL_NSEQS;
  *bytes = latent_decode_workspace(L, n_seqs);
  return PSW_OK;
}

int latent_norm_rope_cache_write(const psw_latent_t* layer, const psw_latent_norm_t* norm,
                                 const void* ckv, int64_t ckv_stride, const void* q_rope,
                                 int64_t q_token_stride, int64_t q_head_stride,
                                 const int32_t* cu_new, const int32_t* past_lens, int32_t n_seqs,
                                 int32_t n_new_total, const psw_pages_t* pages, void* q_rope_out,
                                 int64_t qo_token_stride, int64_t qo_head_stride, void* pool,
                                 psw_stream_t stream) {
  return write_rows(layer, norm, ckv, ckv_stride, q_rope, q_token_stride, q_head_stride, cu_new,
                    past_lens, n_seqs, n_new_total, pages, q_rope_out, qo_token_stride,
                    qo_head_stride, pool, nullptr, stream);
}

int latent_norm_rope_cache_write_fp8(const psw_latent_t* layer, const psw_latent_norm_t* norm,
                                     const void* ckv, int64_t ckv_stride, const void* q_rope,
                                     int64_t q_token_stride, int64_t q_head_stride,
                                     const int32_t* cu_new, const int32_t* past_lens,
                                     int32_t n_seqs, int32_t n_new_total,
                                     const psw_pages_t* pages, void* q_rope_out,
                                     int64_t qo_token_stride, int64_t qo_head_stride, void* pool8,
                                     float* row_scale, psw_stream_t stream) {
  if (row_scale == nullptr) return PSW_ENULL;
  return write_rows(layer, norm, ckv, ckv_stride, q_rope, q_token_stride, q_head_stride, cu_new,
                    past_lens, n_seqs, n_new_total, pages, q_rope_out, qo_token_stride,
                    qo_head_stride, pool8, row_scale, stream);
}

int attn_decode_latent(const psw_latent_t* layer, const void* q, const void* pool,
                       const psw_pages_t* pages, const int32_t* seq_lens, int32_t n_seqs,
                       void* out, float* lse, void* ws, size_t ws_bytes, psw_stream_t stream) {
  return decode(layer, q, pool, nullptr, pages, seq_lens, n_seqs, out, lse, ws, ws_bytes, stream);
}

int attn_decode_latent_fp8(const psw_latent_t* layer, const void* q, const void* pool8,
                           const float* row_scale, const psw_pages_t* pages,
                           const int32_t* seq_lens, int32_t n_seqs, void* out, float* lse,
                           void* ws, size_t ws_bytes, psw_stream_t stream) {
  if (row_scale == nullptr) return PSW_ENULL;
  return decode(layer, q, pool8, row_scale, pages, seq_lens, n_seqs, out, lse, ws, ws_bytes,
                stream);
}

int latent_kv_expand(const psw_latent_t* layer, const void* pool, const psw_pages_t* pages,
                     const int32_t* cu_k, const int32_t* k_first, int32_t n_seqs,
                     int32_t n_k_total, const void* w, void* kv, void* k_rope,
                     psw_stream_t stream) {
  return expand(layer, pool, nullptr, pages, cu_k, k_first, n_seqs, n_k_total, w, kv, k_rope,
                stream);
}

int latent_kv_expand_fp8(const psw_latent_t* layer, const void* pool8, const float* row_scale,
                         const psw_pages_t* pages, const int32_t* cu_k, const int32_t* k_first,
                         int32_t n_seqs, int32_t n_k_total, const void* w, void* kv, void* k_rope,
                         psw_stream_t stream) {
  if (row_scale == nullptr) return PSW_ENULL;
  return expand(layer, pool8, row_scale, pages, cu_k, k_first, n_seqs, n_k_total, w, kv, k_rope,
                stream);
}

int attn_prefill_latent(const psw_latent_t* layer, const void* q, const int32_t* cu_q,
                        const int32_t* past_lens, int32_t n_seqs, int32_t n_q_total,
                        int32_t max_q_len, const void* kv, const void* k_rope,
                        const int32_t* cu_k, const int32_t* k_first, int32_t n_k_total, void* out,
                        float* lse, psw_stream_t stream) {
  LatentArgs L;
  int rc = check_latent(layer, &L);
  if (rc != PSW_OK) return rc;
  if (q == nullptr || cu_q == nullptr || past_lens == nullptr || cu_k == nullptr ||
      out == nullptr || (n_k_total != 0 && (kv == nullptr || k_rope == nullptr)))
    return PSW_ENULL;
  if (n_seqs < 0 || n_seqs > 65535) return PSW_EINVAL_NSEQS;
  if (n_q_total < 0 || max_q_len < 0 || n_k_total < 0) return PSW_ECAPACITY;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(k_rope, 16) || !aligned(out, 16) ||
      !aligned(lse, 4))
    return PSW_EALIGN;
  if (n_seqs == 0 || max_q_len == 0 || n_q_total == 0) return PSW_OK;
  DeviceInfo info;
  int32_t* err;
  if ((rc = ready(&info, &err)) != PSW_OK) return rc;
  return launch_latent_prefill(L, q, cu_q, past_lens, n_seqs, n_q_total, max_q_len, kv, k_rope,
                               cu_k, k_first, n_k_total, out, lse, info.num_sms, err,
                               reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
