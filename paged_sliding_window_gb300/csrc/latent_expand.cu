// latent_expand.cu -- cached latent rows read back from their pages and
// expanded to every head's key and value components:
//   kv[t][h][e] = sum_l c_l w[h][e][l],  k_rope[t] = r.
// 16 rows per CTA and one head: the rows in shared memory as fp32, one output
// component per thread.
#include <cuda_fp8.h>

#include "latent.cuh"

namespace psw {
namespace {

constexpr int kTile = 16;

template <int LAT>
__global__ void __launch_bounds__(kLatentKv)
latent_expand_kernel(const LatentPages pages, const int32_t* __restrict__ cu_k,
                     const int32_t* __restrict__ k_first, int n_seqs, int n_k, int heads,
                     const __nv_bfloat16* __restrict__ w, __nv_bfloat16* __restrict__ kv,
                     __nv_bfloat16* __restrict__ k_rope, int32_t* err) {
  constexpr int kRow = LAT + kLatentRope;
  __shared__ float s[kTile][kRow];
  const int t0 = blockIdx.x * kTile, head = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = min(kTile, min(n_k, __ldg(cu_k + n_seqs)) - t0);
  if (rows <= 0) return;
  for (int i = warp; i < rows; i += 8) {
    int b, start;
    int64_t slot = -1;
    int32_t bits = 0;
    if (!lat::owner_of(cu_k, n_seqs, t0 + i, lane, b, start)) {
      bits = PSW_DEVERR_LENGTH;
    } else {
      const int first = k_first != nullptr ? __ldg(k_first + b) : 0;
      const int64_t pos = static_cast<int64_t>(first) + (t0 + i - start);
      if (first < 0) {
        bits = PSW_DEVERR_LENGTH;
      } else if (pos / kBlockSize >= pages.max_blocks) {
        bits = PSW_DEVERR_CAPACITY;
      } else {
        const int32_t blk =
            __ldg(pages.block_table + static_cast<int64_t>(b) * pages.max_blocks + pos / kBlockSize);
        if (blk < 0 || blk >= pages.num_blocks) bits = PSW_DEVERR_BLOCK_ID;
        else slot = static_cast<int64_t>(blk) * kBlockSize + pos % kBlockSize;
      }
    }
    if (bits != 0 && lane == 0) flag_error(err, bits);
    for (int e = lane; e < kRow; e += 32) {
      float x = 0.f;
      if (slot >= 0) {
        if (pages.row_scale != nullptr) {
          __nv_fp8_e4m3 c;
          c.__x = static_cast<const uint8_t*>(pages.pool)[slot * kRow + e];
          x = static_cast<float>(c) * pages.row_scale[slot];
        } else {
          x = __bfloat162float(static_cast<const __nv_bfloat16*>(pages.pool)[slot * kRow + e]);
        }
      }
      s[i][e] = x;
    }
  }
  __syncthreads();
  const int e = threadIdx.x;
  float acc[kTile];
#pragma unroll
  for (int i = 0; i < kTile; ++i) acc[i] = 0.f;
  const __nv_bfloat16* wr = w + (static_cast<int64_t>(head) * kLatentKv + e) * LAT;
  for (int l = 0; l < LAT; l += 8) {
    float x[8];
    lat::unpack8(__ldg(reinterpret_cast<const uint4*>(wr + l)), x);
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int i = 0; i < kTile; ++i) acc[i] = fmaf(s[i][l + d], x[d], acc[i]);
  }
  for (int i = 0; i < kTile; ++i) {
    if (i >= rows) break;
    kv[(static_cast<int64_t>(t0 + i) * heads + head) * kLatentKv + e] = __float2bfloat16_rn(acc[i]);
    if (head == 0 && e < kLatentRope)
      k_rope[static_cast<int64_t>(t0 + i) * kLatentRope + e] = __float2bfloat16_rn(s[i][LAT + e]);
  }
}

}  // namespace

int launch_latent_expand(const LatentArgs& L, const LatentPages& pages, const int32_t* cu_k,
                         const int32_t* k_first, int n_seqs, int n_k_total, const void* w,
                         void* kv, void* k_rope, int num_sms, int32_t* err, cudaStream_t stream) {
  const dim3 grid((n_k_total + kTile - 1) / kTile, L.n_heads);
  auto* kernel = L.latent == 512 ? latent_expand_kernel<512> : latent_expand_kernel<256>;
  kernel<<<grid, kLatentKv, 0, stream>>>(pages, cu_k, k_first, n_seqs, n_k_total, L.n_heads,
                                         static_cast<const __nv_bfloat16*>(w),
                                         static_cast<__nv_bfloat16*>(kv),
                                         static_cast<__nv_bfloat16*>(k_rope), err);
  return cudaGetLastError() == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

}  // namespace psw
