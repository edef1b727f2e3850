// latent_cache.cu -- the step before latent attention, fused: RMS-norm of the
// new tokens' latents, rotation of the shared key part and of the queries'
// rotary part, and the cache write into bf16 or FP8 pages.
//
// Mathematics, for token t of sequence b at pos = past_b + t - cu_new[b]:
//   row = [ c / sqrt(mean(c^2) + eps) * w | rot(r, pos) ],
//   rot turns (x_i, x_{i+32}) by pos * theta^(-i/32), i < 32,
// rounded once: to bf16, or (FP8 pages) to E4M3 codes of row * 448 / amax with
// the fp32 scale amax / 448. Sums, norms and angles are fp32.
//
// The step is bound by memory on a chunk and by its chain of dependent loads
// (offsets, then the table entry) on a decode batch. A warp's unit is a
// token's cache row or eight (of many: sixteen) of its query heads, so that a
// decode batch spreads over many SMs, and the unit's own loads are issued before
// the chain starts. The 32 angles of a token sit one per lane; the query lanes, which
// hold 8 + 8 values each for 16-byte accesses, fetch theirs by shuffles.
//
// Measured (latent 512, in a graph): 64 tokens of 16 heads 3.9 us; 4096 tokens 6.9
// us, 26 MB read and written (3.8 TB/s); 6900 tokens of 32 heads into FP8 pages
// 16.0 us, 66 MB (4.1 TB/s, 61 % of the measured copy rate). A single call takes the
// 20 to 30 us that the host needs for it. What is left: a warp's loads are in flight for
// part of the time only. It finds its token, computes and stores before it asks for the
// next unit's values, and each unit of a token finds position and angles again.
#include <math.h>

#include "latent.cuh"

namespace psw {
namespace {

constexpr int kWarps = 4;
constexpr int kGroup = 8;  // query heads that a warp turns at once
constexpr int kCtas = 8;   // per SM
constexpr float kLeastRow = 0x1p-117f;  // FP8: largest value of a row that is not taken for zeros

struct Freqs {
  double f[kLatentRope / 2];   // theta^(-i / 32), for positions from 2^24 on
  float2 f2[kLatentRope / 2];  // the same as a float and the float of the rest
};

// Angle pos * f of one pair, as (cos, sin). Below 2^24 pos is exact in fp32:
// the product with the two-float frequency is formed with its rounding error
// (an FMA returns it), reduced by a three-float pi / 2 (Cody-Waite: every FMA
// multiplies exactly), and once more because above 2^22 the quotient may be
// off by one or two. Beyond, in double. Sine and cosine on [-pi/4, pi/4] are
// the Taylor polynomials through x^9 and x^8 (2.5e-8 at most), the quadrant
// swaps and signs them.
__device__ __forceinline__ void turn_of(int pos, float2 fq, double fd, float& cs, float& sn) {
  constexpr float kP1 = 1.5707963705062866f, kP2 = -4.3711388286737929e-8f,
                  kP3 = -1.7151245100058819e-15f, kTwoOverPi = 0.63661974668502808f;
  float x;
  int qd;
  if (pos < (1 << 24)) {
    const float pf = static_cast<float>(pos);
    const float ph = pf * fq.x;
    const float pl = fmaf(pf, fq.y, fmaf(pf, fq.x, -ph));
    const float n1 = rintf(ph * kTwoOverPi);
    x = fmaf(-n1, kP3, fmaf(-n1, kP2, fmaf(-n1, kP1, ph))) + pl;
    const float n2 = rintf(x * kTwoOverPi);
    x = fmaf(-n2, kP2, fmaf(-n2, kP1, x));
    qd = static_cast<int>(n1) + static_cast<int>(n2);
  } else {
    constexpr double kHalfPiHi = 1.5707963267948966, kHalfPiLo = 6.123233995736766e-17;
    const double a = static_cast<double>(pos) * fd;
    const double n1 = rint(a * (1.0 / kHalfPiHi));
    x = static_cast<float>(fma(-n1, kHalfPiLo, fma(-n1, kHalfPiHi, a)));
    qd = static_cast<int>(static_cast<int64_t>(n1) & 3);
  }
  const float x2 = x * x;
  float sp = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
  sp = fmaf(x2, sp, 1.f / 120.f);
  sp = fmaf(x2, sp, -1.f / 6.f);
  const float sx = fmaf(x * x2, sp, x);
  float cp = fmaf(x2, 1.f / 40320.f, -1.f / 720.f);
  cp = fmaf(x2, cp, 1.f / 24.f);
  cp = fmaf(x2, cp, -0.5f);
  const float cx = fmaf(x2, cp, 1.f);
  const float s0 = (qd & 1) ? cx : sx, c0 = (qd & 1) ? sx : cx;
  sn = (qd & 2) ? -s0 : s0;
  cs = ((qd + 1) & 2) ? -c0 : c0;
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float k) {
  return lat::e4m3_pair(a * k, b * k) | lat::e4m3_pair(c * k, d * k) << 16;
}

template <int LAT, bool FP8, int GROUPS>
__global__ void __launch_bounds__(kWarps * 32, kCtas)
latent_write_kernel(const __grid_constant__ Freqs freqs, const float* __restrict__ weight,
                    float eps, const __nv_bfloat16* __restrict__ ckv, int64_t ckv_stride,
                    const LatentRows q, int heads, const int32_t* __restrict__ cu_new,
                    const int32_t* __restrict__ past_lens, int n_seqs, int n_new_total,
                    const int32_t* __restrict__ block_table, int max_blocks, int64_t num_blocks,
                    void* __restrict__ pool, float* __restrict__ row_scale, int32_t* err) {
  constexpr int kRow = LAT + kLatentRope, kVecs = LAT / 256, kHalf = kLatentRope / 2;
  constexpr int kUnitHeads = kGroup * GROUPS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ float2 s_f2[kHalf];
  if (threadIdx.x < kHalf) s_f2[threadIdx.x] = freqs.f2[threadIdx.x];
  __syncthreads();
  const int named = __ldg(cu_new + n_seqs), total = min(named, n_new_total);
  if (named > n_new_total && blockIdx.x == 0 && threadIdx.x == 0)
    flag_error(err, PSW_DEVERR_LENGTH);
  const int per_token = 1 + (q.in != nullptr ? (heads + kUnitHeads - 1) / kUnitHeads : 0);
  const int64_t units = static_cast<int64_t>(total) * per_token;
  // unit u on CTA u mod grid: the few units of a decode batch meet every SM
  for (int64_t u = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x; u < units;
       u += static_cast<int64_t>(kWarps) * gridDim.x) {
    const int t = static_cast<int>(u / per_token), part = static_cast<int>(u - static_cast<int64_t>(t) * per_token);
    // this unit's values
    uint4 v[GROUPS][2];
    float r0 = 0.f, r1 = 0.f;
    const int head = (part - 1) * kUnitHeads + (lane >> 2);  // of the first group
    if (part == 0) {
      const __nv_bfloat16* src = ckv + t * ckv_stride;
#pragma unroll
      for (int c = 0; c < kVecs; ++c) v[0][c] = __ldg(reinterpret_cast<const uint4*>(src + c * 256) + lane);
      r0 = __bfloat162float(src[LAT + lane]);
      r1 = __bfloat162float(src[LAT + kHalf + lane]);
    } else {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(q.in) + t * q.in_token +
                                 head * q.in_head + (lane & 3) * 8;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        if (head + g * kGroup >= heads) break;
        v[g][0] = *reinterpret_cast<const uint4*>(src + g * kGroup * q.in_head);
        v[g][1] = *reinterpret_cast<const uint4*>(src + g * kGroup * q.in_head + kHalf);
      }
    }
    int b, start;
    if (!lat::owner_of(cu_new, n_seqs, t, lane, b, start)) {
      if (lane == 0) flag_error(err, PSW_DEVERR_LENGTH);
      continue;
    }
    const int past = __ldg(past_lens + b);
    const int64_t pos64 = static_cast<int64_t>(past) + (t - start);
    if (past < 0 || pos64 > 0x7fffffffLL) {
      if (lane == 0) flag_error(err, PSW_DEVERR_LENGTH);
      continue;
    }
    const int pos = static_cast<int>(pos64);
    int64_t slot = -1;
    if (part == 0) {
      const int page = pos / kBlockSize;
      if (page < max_blocks) {
        const int32_t blk = __ldg(block_table + static_cast<int64_t>(b) * max_blocks + page);
        if (blk >= 0 && blk < num_blocks)
          slot = static_cast<int64_t>(blk) * kBlockSize + pos % kBlockSize;
        else if (lane == 0)
          flag_error(err, PSW_DEVERR_BLOCK_ID);
      } else if (lane == 0) {
        flag_error(err, PSW_DEVERR_CAPACITY);
      }
      if (slot < 0) continue;
    }
    float cs, sn;
    turn_of(pos, s_f2[lane], freqs.f[lane], cs, sn);
    if (part > 0) {
      float c[8], sine[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = __shfl_sync(0xffffffffu, cs, (lane & 3) * 8 + e);
        sine[e] = __shfl_sync(0xffffffffu, sn, (lane & 3) * 8 + e);
      }
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(q.out) + t * q.out_token +
                           head * q.out_head + (lane & 3) * 8;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        if (head + g * kGroup >= heads) break;
        float lo[8], hi[8], olo[8], ohi[8];
        lat::unpack8(v[g][0], lo);
        lat::unpack8(v[g][1], hi);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          olo[e] = fmaf(lo[e], c[e], -(hi[e] * sine[e]));
          ohi[e] = fmaf(hi[e], c[e], lo[e] * sine[e]);
        }
        *reinterpret_cast<uint4*>(dst + g * kGroup * q.out_head) = lat::pack8(olo);
        *reinterpret_cast<uint4*>(dst + g * kGroup * q.out_head + kHalf) = lat::pack8(ohi);
      }
      continue;
    }
    float y[kVecs][8], ss = 0.f;
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
      lat::unpack8(v[0][c], y[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[c][e], y[c][e], ss);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const float inv = rsqrtf(ss * (1.f / LAT) + eps);
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
      float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (weight != nullptr) {
        const float4* wp = reinterpret_cast<const float4*>(weight + c * 256 + lane * 8);
        const float4 a = __ldg(wp), d = __ldg(wp + 1);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        w[4] = d.x, w[5] = d.y, w[6] = d.z, w[7] = d.w;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) y[c][e] = y[c][e] * inv * w[e];
    }
    const float k0 = fmaf(r0, cs, -(r1 * sn)), k1 = fmaf(r1, cs, r0 * sn);
    if (!FP8) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(pool) + slot * kRow;
#pragma unroll
      for (int c = 0; c < kVecs; ++c) reinterpret_cast<uint4*>(dst + c * 256)[lane] = lat::pack8(y[c]);
      dst[LAT + lane] = __float2bfloat16_rn(k0);
      dst[LAT + kHalf + lane] = __float2bfloat16_rn(k1);
    } else {
      float amax = fmaxf(fabsf(k0), fabsf(k1));
#pragma unroll
      for (int c = 0; c < kVecs; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[c][e]));
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
      // (448 / amax and amax / 448 are fp32 numbers from here on; below, a zero row)
      if (amax < kLeastRow) amax = 0.f;
      const float k = amax > 0.f ? __fdiv_rn(448.f, amax) : 0.f;
      uint8_t* dst = static_cast<uint8_t*>(pool) + slot * kRow;
#pragma unroll
      for (int c = 0; c < kVecs; ++c)
        reinterpret_cast<uint2*>(dst + c * 256)[lane] =
            make_uint2(codes4(y[c][0], y[c][1], y[c][2], y[c][3], k),
                       codes4(y[c][4], y[c][5], y[c][6], y[c][7], k));
      const uint32_t kk = codes4(k0, k1, 0.f, 0.f, k);
      dst[LAT + lane] = static_cast<uint8_t>(kk);
      dst[LAT + kHalf + lane] = static_cast<uint8_t>(kk >> 8);
      if (lane == 0) row_scale[slot] = __fdiv_rn(amax, 448.f);
    }
  }
}

}  // namespace

int launch_latent_write(const LatentArgs& L, float theta, float eps, const float* weight,
                        const void* ckv, int64_t ckv_stride, const LatentRows& q,
                        const int32_t* cu_new, const int32_t* past_lens, int n_seqs,
                        int n_new_total, const LatentPages& pages, void* pool, float* row_scale,
                        int num_sms, int32_t* err, cudaStream_t stream) {
  Freqs fr;
  const double log_theta = log(static_cast<double>(theta));
  for (int i = 0; i < kLatentRope / 2; ++i) {
    fr.f[i] = exp(-2.0 * i / kLatentRope * log_theta);
    const float hi = static_cast<float>(fr.f[i]);
    fr.f2[i] = make_float2(hi, static_cast<float>(fr.f[i] - static_cast<double>(hi)));
  }
  // Two groups of heads to a unit (twice the bytes in flight, the angles once) where
  // all warps have two units or more: 7.5 -> 6.9 us for 4096 tokens of 16 heads, 18.7
  // -> 16.0 for 6900 of 32. Four (at any number of CTAs): 7.1 and 15.6 at best.
  // Fewer units are spread over as many warps as there are.
  const int64_t units = static_cast<int64_t>(n_new_total) * (1 + (L.n_heads + kGroup - 1) / kGroup);
  const int grid = num_sms * kCtas;
  const bool many = q.in != nullptr && L.n_heads > kGroup &&
                    units > 2 * static_cast<int64_t>(grid) * kWarps;
  const auto* x = static_cast<const __nv_bfloat16*>(ckv);
#define PSW_LAUNCH(LAT_, FP8_, G_)                                                              \
  latent_write_kernel<LAT_, FP8_, G_><<<grid, kWarps * 32, 0, stream>>>(                        \
      fr, weight, eps, x, ckv_stride, q, L.n_heads, cu_new, past_lens, n_seqs, n_new_total,     \
      pages.block_table, pages.max_blocks, pages.num_blocks, pool, row_scale, err)
#define PSW_PICK(LAT_, FP8_)     \
  do {                           \
    if (many)                    \
      PSW_LAUNCH(LAT_, FP8_, 2); \
    else                         \
      PSW_LAUNCH(LAT_, FP8_, 1); \
  } while (0)
  if (L.latent == 512) {
    if (row_scale != nullptr) PSW_PICK(512, true);
    else PSW_PICK(512, false);
  } else {
    if (row_scale != nullptr) PSW_PICK(256, true);
    else PSW_PICK(256, false);
  }
#undef PSW_PICK
#undef PSW_LAUNCH
  return cudaGetLastError() == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

}  // namespace psw
