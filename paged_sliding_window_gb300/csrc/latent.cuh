// latent.cuh -- device pieces shared by the latent-attention kernels.
// Library-internal.
#pragma once

#include <cuda_fp8.h>

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

// tanh, for the softcap of scores cap tanh(s / cap). From t = e^-2|y|, 1 - t over 1 + t is
// good to 2^-22, and a score to that of the cap: 2^-13 up to a cap of kNearCap. Beyond,
// where the cap is far above the scores, they have to stay as near to s as fp32 is: up to
// |y| = 1/4 the odd Taylor polynomial through y^7 (what follows is 3.3e-7 of it at most),
// above it 1 - t keeps all but two of its bits.
constexpr float kNearCap = 512.f;
constexpr float kTanhSmall = 0.25f;
__device__ __forceinline__ float tanh_small_over(float y2) {  // tanh(y) / y
  return fmaf(y2, fmaf(y2, fmaf(y2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
}
__device__ __forceinline__ float tanh_large(float y) {
  const float t = ex2_approx(-2.f * kLog2e * fabsf(y));
  return copysignf(__fdividef(1.f - t, 1.f + t), y);
}
__device__ __forceinline__ float tanh_of(float y) {
  return fabsf(y) <= kTanhSmall ? y * tanh_small_over(y * y) : tanh_large(y);
}

// 2-D view of a pool (or of any rows) as the 3-D map's first two dimensions:
// one box of shared memory rows at (x, y); z selects within a third dimension.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                        int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// ---- clusters: the rank of this CTA, a barrier of all their threads.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

// ---- pairs of CTAs (clusters of two) whose tensor cores work on one product of
// 256 rows: rows 128 r .. of A and D are those of the CTA of rank r, in the same
// places of its own memories, and so is half of B's N. One thread of rank 0
// issues; tensor memory is taken and freed by both.
__device__ __forceinline__ void alloc_pair(uint32_t* smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(smem_dst)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void mma_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this place in both CTAs once this thread's products of
// the pair have ended.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// Arrives on rank 0's barrier at this place. What it announces lies in this CTA's
// own tensor and shared memory and is read there by its own tensor core, so that
// no write to global memory has to be ordered for the other CTA's threads (a release
// for the whole cluster takes ~1000 cycles).
__device__ __forceinline__ void arrive_at_first(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// ---- work of clusters of the grid that have not started: asks for one of them (the
// answer, 16 bytes, comes to `dst`, in a pair to both CTAs, and is counted on `bar`
// there), and reads the answer: its first CTA's index, or -1 if none is left, after
// which no other may be asked for.
template <bool PAIR>
__device__ __forceinline__ void ask_for_work(void* dst, uint64_t* bar) {
  if (PAIR)
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
        ".multicast::cluster::all.b128 [%0], [%1];" ::"r"(smem_u32(dst)),
        "r"(smem_u32(bar))
        : "memory");
  else
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
        " [%0], [%1];" ::"r"(smem_u32(dst)),
        "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ int work_given(const void* src) {
  uint32_t given, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
      "ld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
      : "=r"(given), "=r"(x)
      : "r"(smem_u32(src))
      : "memory");
  return given != 0 ? static_cast<int>(x) : -1;
}

// Plain copy of `bytes` (a multiple of 16; both addresses 16-byte aligned) into
// shared memory, counted on `bar`. (A tensor copy's destination would have to be
// 128-byte aligned.)
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Asynchronous 16-byte copy into shared memory (this thread's group); with
// `bytes` 0 nothing is read and the destination becomes zero.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
// Two floats as E4M3 codes (to nearest even, saturating), and back.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3_values(uint32_t pair) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// D[tmem] (+)= A[smem] * B[smem] on E4M3 operands, fp32 accumulators.
__device__ __forceinline__ void mma_ss_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f8f6f4 with E4M3 A and B (format 0), fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, int a_mn, int b_mn) {
  return tc::idesc_bf16_f32(M, N, a_mn, b_mn) & ~((7u << 7) | (7u << 10));
}

// Whether `p` holds for any of `threads` threads of named barrier `id`.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t threads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "barrier.cta.red.or.pred b, %2, %3, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// True on one lane of the (converged) warp. Code that issues MMAs stays converged
// around it, so that descriptors live in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

// 16 lanes x 256 bits, 2 repetitions (16 columns): register 4k + e of thread t
// holds lane t/4 (e = 0, 1) or lane 8 + t/4 (e = 2, 3), column 8k + 2 (t mod 4)
// + (e mod 2), as tc::ld16x256_x4.
__device__ __forceinline__ void ld16x256_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

// 32 lanes x 32 bits of one column.
__device__ __forceinline__ void ld1(uint32_t taddr, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}
__device__ __forceinline__ void st1(uint32_t taddr, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}

// Maximum over a warp (NaN inputs are ignored).
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

}  // namespace lat
}  // namespace psw
