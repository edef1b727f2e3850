// latent.cuh -- device pieces shared by the latent-attention kernels.
// Library-internal.
#pragma once

#include "psw_internal.h"
#include "ptx.cuh"

namespace psw {
namespace lat {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The sequence of flat row t, found by a whole warp: the largest b below
// n_seqs with cu[b] <= t. Each round the lanes probe the open range at 31
// evenly spaced offsets (one coalesced load) and a ballot narrows it to one
// stride; the round of stride 1 also yields the ends of the sequence. False
// when t lies outside [cu[b], cu[b + 1]) (offsets that are not monotone, or a
// row before the first sequence). Every lane returns the same values.
__device__ __forceinline__ bool owner_of(const int32_t* __restrict__ cu, int n_seqs, int t,
                                         int lane, int& b, int& start) {
  int lo = 0, hi = n_seqs;
  while (hi > lo) {
    const int step = (hi - lo + 30) / 31;
    const int idx = lo + lane * step;
    const int c = idx <= hi ? __ldg(cu + idx) : 0;
    const unsigned m = __ballot_sync(0xffffffffu, idx < hi && c <= t);
    if (m == 0) return false;
    const int h = 31 - __clz(static_cast<int>(m));
    if (step == 1) {  // h <= 30: lane h + 1 holds cu[b + 1]
      b = lo + h;
      start = __shfl_sync(0xffffffffu, c, h);
      return t < __shfl_sync(0xffffffffu, c, h + 1);
    }
    lo += h * step;
    hi = min(hi, lo + step);
  }
  return false;
}

__device__ __forceinline__ void unpack8(const uint4& r, float (&y)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[2 * e] = __uint_as_float(w[e] << 16);
    y[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                    pack_bf16x2(y[6], y[7]));
}

}  // namespace lat
}  // namespace psw
