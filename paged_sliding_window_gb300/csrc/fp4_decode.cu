// fp4_decode.cu -- attention of one token per sequence over 4-bit pages.
//
//   s_j = scale * <q, K_j>, capped;  out = sum_j softmax(s)_j V_j
// over the keys that window and length leave, K_j and V_j being code * block
// scale * tensor scale.
#include "fp4.cuh"
#include "latent.cuh"

namespace psw {
namespace {

using fp4::Page;

constexpr int kWarps = 8;

// Simple form: one CTA per (sequence, KV head, up to 8 query heads); its warps
// take the visible tokens in turn, each lane HD / 32 values of a row.
template <int HD>
__global__ void __launch_bounds__(kWarps * 32)
fp4_decode_kernel(const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ k_pool,
                  const uint8_t* __restrict__ v_pool, const int32_t* __restrict__ table,
                  int max_blocks, int64_t num_blocks, const int32_t* __restrict__ seq_lens,
                  int n_q, int n_kv, int group, int qchunks, int window, float scale,
                  float softcap, float v_scale, __nv_bfloat16* __restrict__ out,
                  float* __restrict__ lse, int32_t* err) {
  constexpr int D = HD / 32;
  extern __shared__ float s_o[];  // [warp][8][HD], then [warp][8] (m, l)
  float2* s_ml = reinterpret_cast<float2*>(s_o + kWarps * 8 * HD);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ups = n_kv * qchunks;
  const int b = blockIdx.x / ups, u = blockIdx.x % ups;
  const int kv = u / qchunks, h0 = kv * group + u % qchunks * 8;
  const int nh = min(8, (kv + 1) * group - h0);
  int len = seq_lens[b];
  if (len < 0 || len > max_blocks * kBlockSize) {
    if (threadIdx.x == 0) flag_error(err, len < 0 ? PSW_DEVERR_LENGTH : PSW_DEVERR_CAPACITY);
    len = len < 0 ? 0 : max_blocks * kBlockSize;
  }
  const int lo = window > 0 && len > window ? len - window : 0;
  float qf[8][D], o[8][D], m[8], l[8];
#pragma unroll
  for (int h = 0; h < 8; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int d = 0; d < D; ++d) {
      o[h][d] = 0.f;
      qf[h][d] = h < nh ? __bfloat162float(
                              q[(static_cast<int64_t>(b) * n_q + h0 + h) * HD + lane * D + d])
                        : 0.f;
    }
  }
  auto row = [&](const uint8_t* page, int r, float (&x)[D]) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int i = lane * D + d;
      const uint32_t byte = page[Page<HD>::unit(r, i >> 5) + ((i & 31) >> 1)];
      const float2 c = fp4::f16x2_to_float2(fp4::codes_f16<0>(byte));
      x[d] = ((i & 1) ? c.y : c.x) * fp4::e4m3_float(page[Page<HD>::scale(r, i >> 4)]);
    }
  };
  for (int pos = lo + warp; pos < len; pos += kWarps) {
    const int32_t blk = table[static_cast<int64_t>(b) * max_blocks + pos / kBlockSize];
    const bool have = blk >= 0 && blk < num_blocks;
    if (!have && lane == 0) flag_error(err, PSW_DEVERR_BLOCK_ID);
    const int64_t at = (static_cast<int64_t>(have ? blk : 0) * n_kv + kv) * Page<HD>::kBytes;
    float x[D];
    row(k_pool + at, pos % kBlockSize, x);
    float p[8], a[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      float s = 0.f;
#pragma unroll
      for (int d = 0; d < D; ++d) s = fmaf(qf[h][d], have ? x[d] : 0.f, s);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      s *= scale;
      if (softcap > 0.f) s = softcap * lat::tanh_of(s / softcap);
      s *= lat::kLog2e;
      const float mn = fmaxf(m[h], s);
      a[h] = exp2f(m[h] - mn);
      p[h] = exp2f(s - mn);
      m[h] = mn;
      l[h] = l[h] * a[h] + p[h];
    }
    if (v_pool != nullptr) row(v_pool + at, pos % kBlockSize, x);
#pragma unroll
    for (int h = 0; h < 8; ++h)
#pragma unroll
      for (int d = 0; d < D; ++d) o[h][d] = fmaf(p[h], have ? x[d] : 0.f, o[h][d] * a[h]);
  }
#pragma unroll
  for (int h = 0; h < 8; ++h) {
#pragma unroll
    for (int d = 0; d < D; ++d) s_o[(warp * 8 + h) * HD + lane * D + d] = o[h][d];
    if (lane == 0) s_ml[warp * 8 + h] = make_float2(m[h], l[h]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nh * HD; i += kWarps * 32) {
    const int h = i / HD, d = i % HD;
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w * 8 + h].x);
    for (int w = 0; w < kWarps && M > -INFINITY; ++w) {
      const float2 ml = s_ml[w * 8 + h];
      const float f = exp2f(ml.x - M);
      L += ml.y * f;
      acc += s_o[(w * 8 + h) * HD + d] * f;
    }
    const int64_t r = static_cast<int64_t>(b) * n_q + h0 + h;
    out[r * HD + d] = __float2bfloat16_rn(len > lo ? acc / L * v_scale : 0.f);
    if (d == 0 && lse != nullptr) lse[r] = len > lo ? (M + log2f(L)) * lat::kLn2 : -INFINITY;
  }
}

}  // namespace

size_t fp4_decode_workspace(const LayerArgs& L, int n_seqs) {
  const size_t slots = kFp4MaxWorkers + static_cast<size_t>(n_seqs) * L.n_kv * L.qchunks();
  const int rows = L.group() < kQHeadsPerUnit ? L.group() : kQHeadsPerUnit;
  return kFp4CounterBytes + slots * rows * (static_cast<size_t>(L.hd) * 4 + 8);
}

int launch_fp4_decode(const LayerArgs& L, const void* q, const void* k_pool, const void* v_pool,
                      const psw_pages_t& pages, const int32_t* seq_lens, int n_seqs, void* out,
                      float* lse, void* ws, float k_scale, float v_scale, int num_sms,
                      int32_t* err, cudaStream_t stream) {
  (void)ws;
  (void)num_sms;
  const int smem = kWarps * 8 * L.hd * 4 + kWarps * 8 * 8;
  auto* fn = L.hd == 256 ? fp4_decode_kernel<256> : fp4_decode_kernel<512>;
  const int rc = set_smem_limit(reinterpret_cast<const void*>(fn), smem);
  if (rc != PSW_OK) return rc;
  fn<<<n_seqs * L.n_kv * L.qchunks(), kWarps * 32, smem, stream>>>(
      static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(k_pool),
      static_cast<const uint8_t*>(v_pool != nullptr || !L.k_eq_v ? v_pool : k_pool),
      pages.block_table, pages.max_blocks_per_seq, pages.num_blocks, seq_lens, L.n_q, L.n_kv,
      L.group(), L.qchunks(), L.window, L.scale * k_scale, L.softcap,
      L.k_eq_v ? k_scale : v_scale, static_cast<__nv_bfloat16*>(out), lse, err);
  return cudaGetLastError() == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

}  // namespace psw
