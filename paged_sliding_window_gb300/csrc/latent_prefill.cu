// latent_prefill.cu -- expanded latent attention of a chunk of queries per
// sequence: keys [kv[:128] | k_rope], values kv[128:].
// One CTA per (16 query rows, head): tiles of 64 keys in shared memory, a warp
// per two rows, the running maximum and sum of the softmax in fp32.
#include "latent.cuh"

namespace psw {
namespace {

constexpr int kRows = 16, kKeys = 32, kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32)
latent_prefill_kernel(const __nv_bfloat16* __restrict__ q, const int32_t* __restrict__ cu_q,
                      const int32_t* __restrict__ past_lens, int n_q, int max_q_len,
                      const __nv_bfloat16* __restrict__ kv,
                      const __nv_bfloat16* __restrict__ k_rope, const int32_t* __restrict__ cu_k,
                      const int32_t* __restrict__ k_first, int n_k, int heads, int window,
                      float scale, float softcap, __nv_bfloat16* __restrict__ out,
                      float* __restrict__ lse, int32_t* err) {
  constexpr int kQk = kLatentNope + kLatentRope;
  __shared__ float s_q[kRows][kQk];
  __shared__ float s_k[kKeys][kQk + 1];
  __shared__ __nv_bfloat16 s_v[kKeys][kLatentV];
  const int b = blockIdx.z, h = blockIdx.y, i0 = blockIdx.x * kRows;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int q0 = cu_q[b], k0 = cu_k[b], past = past_lens[b];
  int nq = cu_q[b + 1] - q0, nk = cu_k[b + 1] - k0;
  const int first = k_first != nullptr ? k_first[b] : 0;
  if (q0 < 0 || nq < 0 || past < 0 || k0 < 0 || nk < 0 || first < 0) {
    if (tid == 0 && i0 == 0 && h == 0) flag_error(err, PSW_DEVERR_LENGTH);
    return;
  }
  if (nq > max_q_len || static_cast<int64_t>(q0) + nq > n_q || static_cast<int64_t>(k0) + nk > n_k) {
    if (tid == 0 && i0 == 0 && h == 0) flag_error(err, PSW_DEVERR_LENGTH);
    nq = min(nq, min(max_q_len, n_q - q0));
    nk = min(nk, n_k - k0);
  }
  if (i0 >= nq) return;
  for (int i = tid; i < kRows * kQk; i += kWarps * 32) {
    const int r = i / kQk, e = i - r * kQk;
    s_q[r][e] = i0 + r < nq ? __bfloat162float(q[((static_cast<int64_t>(q0) + i0 + r) * heads + h) * kQk + e]) : 0.f;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[2][4] = {};
  const int64_t p_last = static_cast<int64_t>(past) + i0 + kRows - 1;
  for (int j0 = 0; j0 < nk && static_cast<int64_t>(first) + j0 <= p_last; j0 += kKeys) {
    if (window > 0 && static_cast<int64_t>(first) + j0 + kKeys - 1 <= static_cast<int64_t>(past) + i0 - window) continue;
    __syncthreads();
    for (int i = tid; i < kKeys * (kLatentKv + kLatentRope); i += kWarps * 32) {
      const int r = i / (kLatentKv + kLatentRope), e = i - r * (kLatentKv + kLatentRope);
      const int64_t row = static_cast<int64_t>(k0) + j0 + r;
      float x = 0.f;
      if (j0 + r < nk)
        x = __bfloat162float(e < kLatentKv ? kv[(row * heads + h) * kLatentKv + e]
                                           : k_rope[row * kLatentRope + e - kLatentKv]);
      if (e < kLatentNope) s_k[r][e] = x;
      else if (e < kLatentKv) s_v[r][e - kLatentNope] = __float2bfloat16_rn(x);
      else s_k[r][e - kLatentKv + kLatentNope] = x;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int r = warp * 2 + w;
      const int64_t p = static_cast<int64_t>(past) + i0 + r, pos = static_cast<int64_t>(first) + j0 + lane;
      float d = 0.f;
      for (int e = 0; e < kQk; ++e) d = fmaf(s_q[r][e], s_k[lane][e], d);
      float s = d * scale;
      if (softcap > 0.f) s = softcap * tanhf(s / softcap);
      const bool seen = j0 + lane < nk && pos <= p && (window == 0 || p - pos < window);
      float mt = seen ? s : -INFINITY;
      for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      mt = fmaxf(mt, m[w]);
      const float base = mt == -INFINITY ? 0.f : mt;
      const float alpha = m[w] == -INFINITY ? 0.f : expf(m[w] - base);
      const float pr = seen ? expf(s - base) : 0.f;
      m[w] = mt;
      l[w] = l[w] * alpha + pr;  // this lane's part
      for (int d4 = 0; d4 < 4; ++d4) acc[w][d4] *= alpha;
      for (int j = 0; j < kKeys; ++j) {
        const float pj = __shfl_sync(0xffffffffu, pr, j);
        if (pj != 0.f)
          for (int d4 = 0; d4 < 4; ++d4) acc[w][d4] = fmaf(pj, __bfloat162float(s_v[j][d4 * 32 + lane]), acc[w][d4]);
      }
    }
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int i = i0 + warp * 2 + w;
    float lt = l[w];
    for (int o = 16; o > 0; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
    if (i >= nq) continue;
    const int64_t row = (static_cast<int64_t>(q0) + i) * heads + h;
    for (int d4 = 0; d4 < 4; ++d4)
      out[row * kLatentV + d4 * 32 + lane] = __float2bfloat16_rn(lt == 0.f ? 0.f : acc[w][d4] / lt);
    if (lse != nullptr && lane == 0) lse[row] = lt == 0.f ? -INFINITY : m[w] + logf(lt);
  }
}

}  // namespace

int launch_latent_prefill(const LatentArgs& L, const void* q, const int32_t* cu_q,
                          const int32_t* past_lens, int n_seqs, int n_q_total, int max_q_len,
                          const void* kv, const void* k_rope, const int32_t* cu_k,
                          const int32_t* k_first, int n_k_total, void* out, float* lse,
                          int num_sms, int32_t* err, cudaStream_t stream) {
  const dim3 grid((max_q_len + kRows - 1) / kRows, L.n_heads, n_seqs);
  latent_prefill_kernel<<<grid, kWarps * 32, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(q), cu_q, past_lens, n_q_total, max_q_len,
      static_cast<const __nv_bfloat16*>(kv), static_cast<const __nv_bfloat16*>(k_rope), cu_k,
      k_first, n_k_total, L.n_heads, L.window, L.scale, L.softcap,
      static_cast<__nv_bfloat16*>(out), lse, err);
  return cudaGetLastError() == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

}  // namespace psw
