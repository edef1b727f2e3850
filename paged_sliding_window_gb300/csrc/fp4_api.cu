// fp4_api.cu -- the entry points of the 4-bit pages and of the tables built on
// the device: argument checks (every error is returned before anything is
// launched) and dispatch to the launchers of fp4_cache.cu, fp4_decode.cu and
// block_tables.cu.
#include <math.h>

#include "psw_internal.h"

using namespace psw;

namespace {

bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

bool tensor_scale_ok(float s) { return s >= 0x1p-60f && s <= 0x1p60f; }  // (false for a NaN)

int ready(DeviceInfo* info, int32_t** err) {
  if (device_info(info) != cudaSuccess || info->cc_major != 10 || info->cc_minor != 3)
    return PSW_EDEVICE;
  *err = device_error_word();
  return PSW_OK;
}

// Pages of all sequences (and `more` entries each), times `units`, must be countable in 32 bits.
bool countable(const psw_pages_t* pages, int32_t n_seqs, int64_t units, int64_t more) {
  return n_seqs * (pages->max_blocks_per_seq + more) <= INT32_MAX / units;
}

}  // namespace

extern "C" {

int block_table_extend(int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* past_lens,
                       const int32_t* new_lens, int32_t n_seqs, const int32_t* free_ids,
                       int32_t n_free, const int32_t* free_pos, int32_t* free_next,
                       int32_t* cu_new, int32_t* seq_lens, int64_t* slots, int32_t n_slots,
                       psw_stream_t stream) {
  if (block_table == nullptr || past_lens == nullptr || new_lens == nullptr ||
      (free_ids == nullptr && n_free > 0) || free_pos == nullptr || free_next == nullptr ||
      cu_new == nullptr || seq_lens == nullptr)
    return PSW_ENULL;
  if (n_seqs < 0) return PSW_EINVAL_NSEQS;
  if (max_blocks_per_seq <= 0 || n_free < 0 || n_slots < 0 ||
      static_cast<int64_t>(max_blocks_per_seq) * kBlockSize > INT32_MAX ||
      static_cast<int64_t>(n_seqs) * max_blocks_per_seq > INT32_MAX)
    return PSW_ECAPACITY;
  if (!aligned(block_table, 4) || !aligned(past_lens, 4) || !aligned(new_lens, 4) ||
      !aligned(free_ids, 4) || !aligned(free_pos, 4) || !aligned(free_next, 4) ||
      !aligned(cu_new, 4) || !aligned(seq_lens, 4) || !aligned(slots, 8))
    return PSW_EALIGN;
  // (without sequences a cursor kept in place stays as it is; a second one has to follow it)
  if (n_seqs == 0 && free_next == free_pos) return PSW_OK;
  DeviceInfo info;
  int32_t* err;
  const int rc = ready(&info, &err);
  if (rc != PSW_OK) return rc;
  return launch_block_table_extend(block_table, max_blocks_per_seq, past_lens, new_lens, n_seqs,
                                   free_ids, n_free, free_pos, free_next, cu_new, seq_lens, slots,
                                   slots != nullptr ? n_slots : 0, err,
                                   reinterpret_cast<cudaStream_t>(stream));
}

int kv_cache_write_fp4(const psw_layer_t* layer, const void* k, const void* v,
                       const int32_t* cu_new, const int32_t* past_lens, int32_t n_seqs,
                       int32_t n_new_total, const psw_pages_t* pages, void* k_pool4,
                       void* v_pool4, float k_scale, float v_scale, psw_stream_t stream) {
  LayerArgs L;
  int rc = check_layer(layer, &L);
  if (rc != PSW_OK) return rc;
  if (k == nullptr || cu_new == nullptr || past_lens == nullptr || k_pool4 == nullptr)
    return PSW_ENULL;
  if ((rc = check_v(L, v)) != PSW_OK) return rc;
  if ((rc = check_v(L, v_pool4)) != PSW_OK) return rc;
  if ((rc = check_pages(pages)) != PSW_OK) return rc;
  if (n_seqs < 0) return PSW_EINVAL_NSEQS;
  if (n_new_total < 0) return PSW_ECAPACITY;
  if (!tensor_scale_ok(k_scale) || !tensor_scale_ok(v_scale)) return PSW_EINVAL_SCALE;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pool4, 16) || !aligned(v_pool4, 16))
    return PSW_EALIGN;
  if (n_seqs == 0 || n_new_total == 0) return PSW_OK;
  DeviceInfo info;
  int32_t* err;
  if ((rc = ready(&info, &err)) != PSW_OK) return rc;
  return launch_fp4_write(L, k, v, cu_new, past_lens, n_seqs, n_new_total, *pages, k_pool4,
                          v_pool4, k_scale, v_scale, err, reinterpret_cast<cudaStream_t>(stream));
}

int kv_cache_read_fp4(const psw_layer_t* layer, const void* k_pool4, const void* v_pool4,
                      const psw_pages_t* pages, const int32_t* first, const int32_t* seq_lens,
                      int32_t n_seqs, const psw_pages_t* out_pages, void* k_pool, void* v_pool,
                      float k_scale, float v_scale, psw_stream_t stream) {
  LayerArgs L;
  int rc = check_layer(layer, &L);
  if (rc != PSW_OK) return rc;
  if (k_pool4 == nullptr || seq_lens == nullptr || k_pool == nullptr) return PSW_ENULL;
  if ((rc = check_v(L, v_pool4)) != PSW_OK) return rc;
  if ((rc = check_v(L, v_pool)) != PSW_OK) return rc;
  if ((rc = check_pages(pages)) != PSW_OK) return rc;
  if ((rc = check_pages(out_pages)) != PSW_OK) return rc;
  if (n_seqs < 0) return PSW_EINVAL_NSEQS;
  if (!tensor_scale_ok(k_scale) || !tensor_scale_ok(v_scale)) return PSW_EINVAL_SCALE;
  if (!aligned(k_pool4, 16) || !aligned(v_pool4, 16) || !aligned(k_pool, 16) ||
      !aligned(v_pool, 16))
    return PSW_EALIGN;
  if (!countable(pages, n_seqs, 1, 0)) return PSW_ECAPACITY;
  if (n_seqs == 0) return PSW_OK;
  DeviceInfo info;
  int32_t* err;
  if ((rc = ready(&info, &err)) != PSW_OK) return rc;
  return launch_fp4_read(L, k_pool4, v_pool4, *pages, first, seq_lens, n_seqs, *out_pages, k_pool,
                         v_pool, k_scale, v_scale, info.num_sms, err,
                         reinterpret_cast<cudaStream_t>(stream));
}

int psw_fp4_workspace_bytes(const psw_layer_t* layer, int32_t n_seqs, size_t* bytes) {
  LayerArgs L;
  const int rc = check_layer(layer, &L);
  if (rc != PSW_OK) return rc;
  if (bytes == nullptr) return PSW_ENULL;
  if (n_seqs < 0) return PSW_EINVAL_NSEQS;
  *bytes = fp4_decode_workspace(L, n_seqs);
  return PSW_OK;
}

int attn_decode_paged_fp4(const psw_layer_t* layer, const void* q, const void* k_pool4,
                          const void* v_pool4, const psw_pages_t* pages, const int32_t* seq_lens,
                          int32_t n_seqs, void* out, float* lse, void* ws, size_t ws_bytes,
                          float k_scale, float v_scale, psw_stream_t stream) {
  LayerArgs L;
  int rc = check_decode_args(layer, q, k_pool4, v_pool4, pages, seq_lens, n_seqs,
                             static_cast<const float*>(out), &L);
  if (rc != PSW_OK) return rc;
  if (!tensor_scale_ok(k_scale) || !tensor_scale_ok(v_scale)) return PSW_EINVAL_SCALE;
  if (!aligned(ws, 16) || !aligned(lse, 4)) return PSW_EALIGN;
  if (!countable(pages, n_seqs, static_cast<int64_t>(L.n_kv) * L.qchunks(), fp4_unit_cost(L.hd)) ||
      static_cast<int64_t>(L.n_kv) * PSW_FP4_PAGE_BYTES(L.hd) > INT32_MAX)
    return PSW_ECAPACITY;
  if (n_seqs == 0) return PSW_OK;
  if (ws == nullptr || ws_bytes < fp4_decode_workspace(L, n_seqs)) return PSW_EWORKSPACE;
  DeviceInfo info;
  int32_t* err;
  if ((rc = ready(&info, &err)) != PSW_OK) return rc;
  return launch_fp4_decode(L, q, k_pool4, v_pool4, *pages, seq_lens, n_seqs, out, lse, ws, k_scale,
                           v_scale, info.num_sms, err, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
