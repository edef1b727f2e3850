// latent_prefill.cu -- expanded latent attention of a chunk of queries per
// sequence: keys [kv[:128] | k_rope], values kv[128:].
//
// Mathematics, per row i at p = past + i and head: over the keys j at positions
// first + j <= p, closer than the window,
//   s_j = softcap(scale <q, k_j>),  out = sum_j softmax(s)_j v_j,
// with the running maximum and sum of an online softmax in fp32. 2 (192 + 128)
// operations per (row, head, key) against 512 bytes of a key per head and
// block of rows: bound by the tensor cores and, before them, by what L2 brings
// to an SM, so a CTA takes 256 rows of one head against every key tile.
//
// Schedule: a CTA has two tiles of 128 rows, A and B. Key tiles of 128 go
// through a ring of 16 KB units (128 keys x 128 B, swizzled): two of key
// components, one of the shared rotary part, two of values. Warp 8 loads. Warp
// 9 issues, in turn for A and B, O += P V of a key tile and S = Q K^T of the
// next: while the softmax of one row tile runs, the tensor cores work for the
// other. P is written over S in tensor memory as bf16 (rounded once; sums are of
// the unrounded values). Warps 0-3 and 4-7 are the softmaxes of A and B, a
// thread per row. The maximum that P is relative to is that of a row's first
// keys; it moves (O rescaled) only when a score exceeds it by 2^64, which P, O
// and the sum have the range for. The longest sequences come first in the grid.
#include <math.h>

#include "latent.cuh"

namespace psw {
namespace lpre {

constexpr int kQk = kLatentNope + kLatentRope;
constexpr int kTile = 128;                    // rows of a row tile, keys of a key tile
constexpr int kUnit = kTile * 128;            // bytes of a ring unit
constexpr int kQChunks = kQk / 64;
constexpr int kQBytes = 2 * kQChunks * kUnit;
constexpr int kUnits = 8;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;
constexpr int kSmemBytes = 1024 + kQBytes + kUnits * kUnit + 2048;
constexpr int kTmemS = 0, kTmemO = 256;       // + 128 for B
constexpr float kLag = 64.f;
constexpr int kRanked = 256;                  // sequences put in order by their length
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

struct Misc {
  uint64_t full[kUnits], empty[kUnits];
  uint64_t q_full[2], s_full[2], p_full[2], pv_done[2], o_full[2];
  uint64_t v_fix, drained;
  uint32_t tmem;
  int32_t abort, seq;
  int32_t len[kRanked];
};
static_assert(sizeof(Misc) <= 2048, "misc block");

// Ring units in the order of use, and each unit's phase. The two units of a
// value tile do not wrap: the last unit is then left out.
struct Ring {
  int pos = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ int take(int n, uint32_t& parity) {
    if (pos + n > kUnits) pos = 0;
    const int s = pos;
    parity = phase >> s;
    phase ^= ((1u << n) - 1u) << s;
    pos = pos + n == kUnits ? 0 : pos + n;
    return s;
  }
};

// What a CTA works on; the same in every thread.
struct Work {
  int q0, rows;         // first row (of q), rows of the CTA
  int k0, nk;           // first key row, keys of the sequence
  int64_t p0, first;    // position of the first row; of the first key
  int lo[2], hi[2];     // key tiles [lo, hi) of A and of B
  int t_lo, t_hi;       // of both
  int j_lo, j_hi;       // keys [j_lo, j_hi) that some row sees
};

__device__ __forceinline__ float tanh_abs(float y) {
  const float t = ex2_approx(-2.f * lat::kLog2e * fabsf(y));
  return copysignf(__fdividef(1.f - t, 1.f + t), y);
}

__global__ void __launch_bounds__(kThreads, 1)
latent_prefill_kernel(const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap kv_map,
                      const __grid_constant__ CUtensorMap rope_map,
                      const int32_t* __restrict__ cu_q, const int32_t* __restrict__ past_lens,
                      int n_seqs, int n_q, int max_q_len, const int32_t* __restrict__ cu_k,
                      const int32_t* __restrict__ k_first, int n_k, int heads, int blocks,
                      int window, float scale, float softcap, __nv_bfloat16* __restrict__ out,
                      float* __restrict__ lse, int32_t* err) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* q_smem = smem;
  uint8_t* ring = smem + kQBytes;
  Misc* ms = reinterpret_cast<Misc*>(ring + kUnits * kUnit);

  // ---- the CTA's sequence, head and block of rows: heads innermost within a
  // sequence's blocks, its last block (the most keys) first
  const int per_seq = heads * blocks;
  const int rank = blockIdx.x / per_seq, sub = blockIdx.x - rank * per_seq;
  const int block = blocks - 1 - sub / heads, head = sub % heads;
  if (warp == kMmaWarp) {
    tc::alloc(&ms->tmem, 512);
    tc::relinquish();
  }
  if (tid == 32 * kLoadWarp) {
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&ms->full[i], 1);
      mbar_init(&ms->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms->q_full[i], 1);
      mbar_init(&ms->s_full[i], 1);
      mbar_init(&ms->p_full[i], 4);
      mbar_init(&ms->pv_done[i], 1);
      mbar_init(&ms->o_full[i], 1);
    }
    mbar_init(&ms->v_fix, 1);
    mbar_init(&ms->drained, 1);
    ms->abort = 0;
    fence_mbar_init();
  }
  // sequence number `rank` by the work of its last row, ties by index
  if (n_seqs <= kRanked) {
    int32_t* s_len = ms->len;
    for (int b = tid; b < n_seqs; b += kThreads) s_len[b] = __ldg(cu_k + b + 1) - __ldg(cu_k + b);
    __syncthreads();
    for (int b = tid; b < n_seqs; b += kThreads) {
      int ahead = 0;
      const int mine = s_len[b];
      for (int o = 0; o < n_seqs; ++o) ahead += s_len[o] > mine || (s_len[o] == mine && o < b);
      if (ahead == rank) ms->seq = b;
    }
  } else if (tid == 0) {
    ms->seq = rank;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = ms->tmem;
  const int b = ms->seq;
  volatile int32_t* abort_flag = &ms->abort;

  Work w;
  bool some = true;
  {
    w.q0 = __ldg(cu_q + b);
    w.k0 = __ldg(cu_k + b);
    int nq = __ldg(cu_q + b + 1) - w.q0;
    w.nk = __ldg(cu_k + b + 1) - w.k0;
    const int past = __ldg(past_lens + b), first = k_first != nullptr ? __ldg(k_first + b) : 0;
    bool bad = false;
    if (w.q0 < 0 || nq < 0 || past < 0 || w.k0 < 0 || w.nk < 0 || first < 0) {
      bad = true;
      nq = 0;
      w.nk = 0;
    }
    if (nq > max_q_len || static_cast<int64_t>(w.q0) + nq > n_q) {
      bad = true;
      nq = max(0, min(nq, min(max_q_len, n_q - w.q0)));
    }
    if (static_cast<int64_t>(w.k0) + w.nk > n_k) {
      bad = true;
      w.nk = max(0, min(w.nk, n_k - w.k0));
    }
    if (bad && tid == 0 && block == 0 && head == 0) flag_error(err, PSW_DEVERR_LENGTH);
    const int i0 = block * 2 * kTile;
    w.rows = min(2 * kTile, nq - i0);
    some = w.rows > 0;
    w.q0 += i0;
    w.p0 = static_cast<int64_t>(past) + i0;
    w.first = first;
    w.t_lo = 0x7fffffff;
    w.t_hi = 0;
    w.j_lo = 0x7fffffff;
    w.j_hi = 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int n = min(kTile, w.rows - g * kTile);
      // keys of the tile's rows: from the window of its first to its last
      const int64_t a = w.p0 + g * kTile;
      const int64_t lo64 = window > 0 ? a - window + 1 - first : 0, hi64 = a + n - first;
      const int lo = static_cast<int>(max(lo64, static_cast<int64_t>(0)));
      const int hi = static_cast<int>(max(min(hi64, static_cast<int64_t>(w.nk)), static_cast<int64_t>(0)));
      const bool any = n > 0 && lo < hi;
      w.lo[g] = any ? lo / kTile : 0;
      w.hi[g] = any ? (hi + kTile - 1) / kTile : 0;
      if (any) {
        w.t_lo = min(w.t_lo, w.lo[g]);
        w.t_hi = max(w.t_hi, w.hi[g]);
        w.j_lo = min(w.j_lo, lo);
        w.j_hi = max(w.j_hi, hi);
      }
    }
  }
  bool ok = true;
  Ring rg;

  if (!some) {
    // no rows: nothing to do
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loads
    const bool one = lat::elect_one();
    uint32_t issued = 0;
    int fixes = 0;
    if (one) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (w.lo[g] >= w.hi[g]) continue;
        mbar_arrive_expect_tx(&ms->q_full[g], kQChunks * kUnit);
        for (int c = 0; c < kQChunks; ++c)
          lat::tma_box(smem_u32(q_smem + (g * kQChunks + c) * kUnit), &q_map, &ms->q_full[g],
                       c * 64, head, w.q0 + g * kTile);
      }
    }
    auto load = [&](int s, uint64_t* bar, const CUtensorMap* map, int x, int y, int z) {
      issued |= 1u << s;
      if (one) lat::tma_box(smem_u32(ring + s * kUnit), map, bar, x, y, z);
    };
    for (int j = w.t_lo; ok && j < w.t_hi; ++j) {
      const int row = w.k0 + j * kTile;
      for (int c = 0; c < 3; ++c) {  // keys: two of the head's components, the rotary part
        uint32_t parity;
        const int s = rg.take(1, parity);
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&ms->empty[s], (parity & 1u) ^ 1u) && *abort_flag == 0);
        if (!ok) break;
        if (one) mbar_arrive_expect_tx(&ms->full[s], kUnit);
        if (c < 2) load(s, &ms->full[s], &kv_map, c * 64, head, row);
        else load(s, &ms->full[s], &rope_map, 0, row, 0);
      }
      if (!ok) break;
      // values; rows of keys that no row sees (other sequences', or anything)
      // must not enter the second product (P is 0 there, but 0 times NaN is not)
      uint32_t parity;
      const int s = rg.take(2, parity);
      for (int c = 0; c < 2; ++c)
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&ms->empty[s + c], (parity >> c & 1u) ^ 1u) && *abort_flag == 0);
      if (!ok) break;
      const int z_lo = max(0, w.j_lo - j * kTile), z_hi = min(kTile, w.j_hi - j * kTile);
      const bool fix = z_lo > 0 || z_hi < kTile;
      if (one) {
        if (fix) mbar_arrive_expect_tx(&ms->v_fix, 2 * kUnit);
        else
          for (int c = 0; c < 2; ++c) mbar_arrive_expect_tx(&ms->full[s + c], kUnit);
      }
      __syncwarp();
      for (int c = 0; c < 2; ++c)
        load(s + c, fix ? &ms->v_fix : &ms->full[s + c], &kv_map, kLatentNope + c * 64, head, row);
      if (fix) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ms->v_fix, fixes & 1));
        ++fixes;
        if (!ok) break;
        for (int i = lane; i < 2 * kTile * 8; i += 32) {
          const int r = (i >> 3) & (kTile - 1);
          if (r < z_lo || r >= z_hi)
            *reinterpret_cast<uint4*>(ring + s * kUnit + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane < 2) mbar_arrive(&ms->full[s + lane]);
      }
    }
    if (!ok && one) {
      *abort_flag = 1;
      flag_error(err, PSW_DEVERR_PIPELINE);
      // copies in flight land before the CTA ends
#pragma unroll
      for (int g = 0; g < 2; ++g)
        if (w.lo[g] < w.hi[g]) mbar_wait(&ms->q_full[g], 0);
      for (int s = 0; s < kUnits; ++s)
        if (issued >> s & 1u) mbar_wait(&ms->full[s], ((rg.phase >> s) & 1u) ^ 1u);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMAs
    const bool one = lat::elect_one();
    constexpr uint32_t id_s = tc::idesc_bf16_f32(kTile, kTile, 0, 0);
    constexpr uint32_t id_o = tc::idesc_bf16_f32(kTile, kLatentV, 0, 1);
    constexpr uint32_t kStep = kUnit >> 4;
    const uint64_t q_desc = tc::smem_desc(smem_u32(q_smem), 16, 1024, tc::kSwizzle128B);
    const uint64_t k_desc = tc::smem_desc(smem_u32(ring), 16, 1024, tc::kSwizzle128B);
    const uint64_t v_desc = tc::smem_desc(smem_u32(ring), kUnit, 1024, tc::kSwizzle128B);
    auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && mbar_wait(bar, parity & 1u); };
    int n[2] = {0, 0};  // S formed for each row tile
    int ks[3], vs = 0;  // units of the key tile at hand, of the value tile
    uint32_t kp[3], vp = 0;
    auto scores = [&](int g) {
      if (n[g] == 0) wait(&ms->q_full[g], 0);
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        wait(&ms->full[ks[c]], kp[c]);
        tc::fence_after();
        const uint64_t kd = k_desc + ks[c] * kStep, qd = q_desc + (g * kQChunks + c) * kStep;
        if (ok && one) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_ss(tmem + kTmemS + g * kTile, qd + k * 2, kd + k * 2, id_s, (c > 0 || k > 0) ? 1u : 0u);
        }
      }
      if (ok && one) tc::commit(&ms->s_full[g]);
      ++n[g];
    };
    auto take_keys = [&]() {
#pragma unroll
      for (int c = 0; c < 3; ++c) ks[c] = rg.take(1, kp[c]);
    };
    auto free_keys = [&]() {
      if (ok && one) {
#pragma unroll
        for (int c = 0; c < 3; ++c) tc::commit(&ms->empty[ks[c]]);
      }
    };
    if (w.t_lo < w.t_hi) {
      take_keys();
#pragma unroll
      for (int g = 0; g < 2; ++g)
        if (w.lo[g] == w.t_lo && w.lo[g] < w.hi[g]) scores(g);
      free_keys();
    }
    for (int j = w.t_lo; ok && j < w.t_hi; ++j) {
      vs = rg.take(2, vp);
      if (j + 1 < w.t_hi) take_keys();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (j >= w.lo[g] && j < w.hi[g]) {
          wait(&ms->p_full[g], n[g] - 1);
          wait(&ms->full[vs], vp);
          wait(&ms->full[vs + 1], vp >> 1);
          tc::fence_after();
          if (ok && one) {
            const uint64_t vd = v_desc + vs * kStep;
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              tc::mma_ts(tmem + kTmemO + g * kLatentV, tmem + kTmemS + g * kTile + k * 8,
                         vd + k * (2048 >> 4), id_o, (j > w.lo[g] || k > 0) ? 1u : 0u);
            tc::commit(&ms->pv_done[g]);
            if (j == w.hi[g] - 1) tc::commit(&ms->o_full[g]);
          }
        }
        if (j + 1 >= w.lo[g] && j + 1 < w.hi[g]) scores(g);
      }
      if (ok && one) {
        tc::commit(&ms->empty[vs]);
        tc::commit(&ms->empty[vs + 1]);
      }
      if (j + 1 < w.t_hi) free_keys();
      ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
    }
    if (one) {
      if (!ok) {
        *abort_flag = 1;
        flag_error(err, PSW_DEVERR_PIPELINE);
      }
      tc::commit(&ms->drained);  // every MMA has ended before tensor memory is freed
      mbar_wait(&ms->drained, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax, epilogue
    const int g = warp >> 2, r = (warp & 3) * 32 + lane, i = g * kTile + r;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + kTmemS + g * kTile;
    const uint32_t o_at = tmem + lanes + kTmemO + g * kLatentV;
    const int64_t p = w.p0 + i;
    const bool cap = softcap > 0.f;
    const float mul = cap ? 1.f : scale * lat::kLog2e;
    const float cap_in = cap ? scale / softcap : 0.f, cap_out = softcap * lat::kLog2e;
    float m = -INFINITY, l = 0.f;
    int n = 0;
    const int t_lo = g == 0 ? w.lo[0] : w.lo[1], t_hi = g == 0 ? w.hi[0] : w.hi[1];
    for (int j = t_lo; j < t_hi; ++j, ++n) {
      // (every decision is the same in the whole warp)
      ok = __all_sync(0xffffffffu, mbar_wait(&ms->s_full[g], n & 1) && *abort_flag == 0);
      if (!ok) break;
      tc::fence_after();
      float x[kTile];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tc::ld32(s_at + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&x[c * 32]));
      tc::wait_ld();
      // this row's visible columns of the tile
      const int64_t at = w.first + static_cast<int64_t>(j) * kTile;
      const int64_t hi64 = min(p - at, static_cast<int64_t>(w.nk - 1 - j * kTile));
      const int64_t lo64 = window > 0 ? p - window + 1 - at : 0;
      const int c_hi = static_cast<int>(max(min(hi64, static_cast<int64_t>(kTile - 1)), static_cast<int64_t>(-1)));
      const int c_lo = static_cast<int>(max(min(lo64, static_cast<int64_t>(kTile)), static_cast<int64_t>(0)));
      if (cap) {
#pragma unroll
        for (int c = 0; c < kTile; ++c) x[c] = cap_out * tanh_abs(x[c] * cap_in);
      }
      if (!__all_sync(0xffffffffu, c_lo <= 0 && c_hi >= kTile - 1)) {
#pragma unroll
        for (int c = 0; c < kTile; ++c) x[c] = c >= c_lo && c <= c_hi ? x[c] : -INFINITY;
      }
      float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int c = 4; c < kTile; c += 8) {
        mx[0] = max3f(mx[0], x[c], x[c + 1]);
        mx[1] = max3f(mx[1], x[c + 2], x[c + 3]);
        if (c + 4 < kTile) {
          mx[2] = max3f(mx[2], x[c + 4], x[c + 5]);
          mx[3] = max3f(mx[3], x[c + 6], x[c + 7]);
        }
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * mul;
      const bool move = top > m + kLag || (m == -INFINITY && top > -INFINITY);
      if (__any_sync(0xffffffffu, move)) {
        // the rows that lag take the tile's maximum; what they have is scaled (a
        // row without keys so far has zeros)
        const float to = move ? top : m;
        const float a = move && m != -INFINITY ? ex2_approx(m - to) : 1.f;
        m = to;
        l *= a;
        if (__any_sync(0xffffffffu, a != 1.f)) {
          ok = __all_sync(0xffffffffu, mbar_wait(&ms->pv_done[g], (n - 1) & 1));
          if (!ok) break;
          tc::fence_after();
#pragma unroll 1
          for (int c = 0; c < kLatentV; c += 16) {
            uint32_t v[16];
            tc::ld16(o_at + c, v);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * a);
            tc::st16(o_at + c, v);
          }
          tc::wait_st();
        }
      }
      const float ref = m == -INFINITY ? 0.f : m;
      const uint64_t mul2 = f2_pack(mul, mul), ref2 = f2_pack(-ref, -ref);
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 z = f2_unpack(f2_fma(f2_pack(x[c * 32 + 2 * e], x[c * 32 + 2 * e + 1]), mul2, ref2));
          const float a0 = ex2_approx(z.x), a1 = ex2_approx(z.y);
          sum[2 * (e & 1)] += a0;
          sum[2 * (e & 1) + 1] += a1;
          pk[e] = pack_bf16x2(a0, a1);
        }
        tc::st16(s_at + c * 16, pk);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->p_full[g]);
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&ms->o_full[g], 0));
    if (ok) {
      tc::fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t row = static_cast<int64_t>(w.q0 + i) * heads + head;
      uint4* dst = reinterpret_cast<uint4*>(out + row * kLatentV);
      const bool mine = i < w.rows;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t v[32];
        if (n > 0) {
          tc::ld32(o_at + c * 32, v);
          tc::wait_ld();
        }
        if (!mine) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y[8];
#pragma unroll
          for (int d = 0; d < 8; ++d) y[d] = l == 0.f ? 0.f : __uint_as_float(v[e * 8 + d]) * inv;
          dst[c * 4 + e] = lat::pack8(y);
        }
      }
      if (mine && lse != nullptr) lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * lat::kLn2;
    } else if (lane == 0) {
      *abort_flag = 1;
      flag_error(err, PSW_DEVERR_PIPELINE);
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tc::dealloc(tmem, 512);
}

}  // namespace lpre

int launch_latent_prefill(const LatentArgs& L, const void* q, const int32_t* cu_q,
                          const int32_t* past_lens, int n_seqs, int n_q_total, int max_q_len,
                          const void* kv, const void* k_rope, const int32_t* cu_k,
                          const int32_t* k_first, int n_k_total, void* out, float* lse,
                          int num_sms, int32_t* err, cudaStream_t stream) {
  using namespace lpre;
  CUtensorMap q_map, kv_map, rope_map;
  const int64_t h = L.n_heads;
  int rc = make_map_3d(&q_map, false, q, {kQk, h, n_q_total}, {2 * kQk, 2 * kQk * h}, {64, 1, kTile});
  if (rc != PSW_OK) return rc;
  if (n_k_total > 0) {
    rc = make_map_3d(&kv_map, false, kv, {kLatentKv, h, n_k_total}, {2 * kLatentKv, 2 * kLatentKv * h},
                     {64, 1, kTile});
    if (rc == PSW_OK)
      rc = make_map_3d(&rope_map, false, k_rope, {kLatentRope, n_k_total, 1},
                       {2 * kLatentRope, 2 * kLatentRope}, {64, kTile, 1});
    if (rc != PSW_OK) return rc;
  } else {
    kv_map = rope_map = q_map;  // no key tile will be loaded
  }
  rc = set_smem_limit(reinterpret_cast<const void*>(latent_prefill_kernel), kSmemBytes);
  if (rc != PSW_OK) return rc;
  const int64_t blocks = (static_cast<int64_t>(max_q_len) + 2 * kTile - 1) / (2 * kTile);
  if (blocks * L.n_heads * n_seqs > 0x7fffffffLL) return PSW_ECAPACITY;
  latent_prefill_kernel<<<static_cast<unsigned>(blocks * L.n_heads * n_seqs), kThreads, kSmemBytes,
                          stream>>>(q_map, kv_map, rope_map, cu_q, past_lens, n_seqs, n_q_total,
                                    max_q_len, cu_k, k_first, n_k_total, L.n_heads,
                                    static_cast<int>(blocks), L.window, L.scale, L.softcap,
                                    static_cast<__nv_bfloat16*>(out), lse, err);
  return cudaGetLastError() == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

}  // namespace psw
