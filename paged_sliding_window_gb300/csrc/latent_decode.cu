// latent_decode.cu -- absorbed latent attention of one token per sequence:
//   s_j = softcap(scale <q, row_j>), out = sum_j softmax(s)_j row_j[:L].
// One CTA per (sequence, head): tiles of 128 keys, one score per thread, the
// running maximum and sum of the softmax, then the values L / 128 per thread.
#include <cuda_fp8.h>

#include "latent.cuh"

namespace psw {
namespace {

constexpr int kThreads = 128;

template <int LAT>
__global__ void __launch_bounds__(kThreads)
latent_decode_kernel(const __nv_bfloat16* __restrict__ q, const LatentPages pages,
                     const int32_t* __restrict__ seq_lens, int heads, int window, float scale,
                     float softcap, __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
                     int32_t* err) {
  constexpr int kRow = LAT + kLatentRope, kPer = LAT / kThreads;
  __shared__ float s_q[kRow], s_p[kThreads], s_red[kThreads];
  __shared__ int64_t s_slot[kThreads];
  const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  int64_t len = seq_lens[b];
  int32_t bits = 0;
  if (len < 0) bits |= PSW_DEVERR_LENGTH, len = 0;
  if (len > static_cast<int64_t>(pages.max_blocks) * kBlockSize)
    bits |= PSW_DEVERR_CAPACITY, len = static_cast<int64_t>(pages.max_blocks) * kBlockSize;
  if (bits != 0 && tid == 0 && h == 0) flag_error(err, bits);
  const int64_t lo = window > 0 && len > window ? len - window : 0;
  for (int e = tid; e < kRow; e += kThreads)
    s_q[e] = __bfloat162float(q[(static_cast<int64_t>(b) * heads + h) * kRow + e]);
  float m = -INFINITY, l = 0.f, acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  auto value = [&](int64_t slot, int e) -> float {
    if (slot < 0) return 0.f;
    if (pages.row_scale != nullptr) {
      __nv_fp8_e4m3 c;
      c.__x = static_cast<const uint8_t*>(pages.pool)[slot * kRow + e];
      return static_cast<float>(c) * pages.row_scale[slot];
    }
    return __bfloat162float(static_cast<const __nv_bfloat16*>(pages.pool)[slot * kRow + e]);
  };
  for (int64_t j0 = lo; j0 < len; j0 += kThreads) {
    __syncthreads();
    const int64_t j = j0 + tid;
    float s = -INFINITY;
    if (j < len) {
      const int32_t blk = pages.block_table[static_cast<int64_t>(b) * pages.max_blocks + j / kBlockSize];
      const bool ok = blk >= 0 && blk < pages.num_blocks;
      if (!ok) flag_error(err, PSW_DEVERR_BLOCK_ID);
      const int64_t slot = ok ? static_cast<int64_t>(blk) * kBlockSize + j % kBlockSize : -1;
      s_slot[tid] = slot;
      float d = 0.f;
      for (int e = 0; e < kRow; ++e) d = fmaf(s_q[e], value(slot, e), d);
      s = d * scale;
      if (softcap > 0.f) s = softcap * tanhf(s / softcap);
    }
    s_red[tid] = s;
    __syncthreads();
    float mt = m;
    for (int i = 0; i < kThreads; ++i) mt = fmaxf(mt, s_red[i]);
    const float base = mt == -INFINITY ? 0.f : mt;
    const float alpha = m == -INFINITY ? 0.f : expf(m - base);
    s_p[tid] = j < len ? expf(s - base) : 0.f;
    __syncthreads();
    m = mt;
    l *= alpha;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] *= alpha;
    const int n = static_cast<int>(min(static_cast<int64_t>(kThreads), len - j0));
    for (int i = 0; i < n; ++i) {
      l += s_p[i];
#pragma unroll
      for (int d = 0; d < kPer; ++d) acc[d] = fmaf(s_p[i], value(s_slot[i], d * kThreads + tid), acc[d]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int d = 0; d < kPer; ++d)
    out[(static_cast<int64_t>(b) * heads + h) * LAT + d * kThreads + tid] =
        __float2bfloat16_rn(acc[d] * inv);
  if (lse != nullptr && tid == 0)
    lse[static_cast<int64_t>(b) * heads + h] = len > 0 ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t latent_decode_workspace(const LatentArgs& L, int n_seqs) { return 256; }

int launch_latent_decode(const LatentArgs& L, const void* q, const LatentPages& pages,
                         const int32_t* seq_lens, int n_seqs, void* out, float* lse, void* ws,
                         int num_sms, int32_t* err, cudaStream_t stream) {
  auto* kernel = L.latent == 512 ? latent_decode_kernel<512> : latent_decode_kernel<256>;
  kernel<<<dim3(n_seqs, L.n_heads), kThreads, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(q), pages, seq_lens, L.n_heads, L.window, L.scale,
      L.softcap, static_cast<__nv_bfloat16*>(out), lse, err);
  return cudaGetLastError() == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

}  // namespace psw
