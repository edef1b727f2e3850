// latent_prefill.cu -- expanded latent attention of a chunk of queries per
// sequence: keys [kv[:128] | k_rope], values kv[128:].
//
// Mathematics, per row i at p = past + i and head: over the keys j at positions
// first + j <= p, closer than the window,
//   s_j = softcap(scale <q, k_j>),  out = sum_j softmax(s)_j v_j,
// with the running maximum and sum of an online softmax in fp32. 2 (192 + 128)
// operations per (row, head, key) against 512 bytes of a key per head and
// block of rows: bound by the tensor cores.
//
// Schedule: two row tiles, A and B, of 128 rows of a CTA, are worked on in turn:
// while the softmax of one runs, the tensor cores work for the other (O += P V of
// a key tile, then S = Q K^T of the next). P is written over S in tensor memory as
// bf16, rounded once; sums are of the unrounded values. That leaves 0.0023 of the output's
// scale against 64 bits, where exact sums rounded to the output's bf16 leave 0.0017. The
// rest of P as a second part would add 128 columns to the 320 that a key tile's products
// have now, 40 % of the time, to take away less than the output's own rounding. Warp 8 loads key tiles
// into stages (swizzled 64-column units), warp 9 issues the products, warps 0-3 and
// 4-7 are the softmaxes of A and B, a thread per row. The maximum that P is
// relative to is that of a row's first keys; it moves (O rescaled) only when a
// score exceeds it by 2^64, which P, O and the sum have the range for.
//
// A product of 128 rows by 128 keys reads as many bytes of shared memory as it
// takes cycles at 128 a cycle, and the key tiles arrive there besides: a CTA by
// itself is bound by its shared memory (573 us for four chunks of 2048 rows after
// 2000 to 16384, 16 heads).
// Chunks of more than 256 rows are therefore done by pairs of CTAs, 512 rows of one
// head (so are shorter ones where there are SMs to spare), whose tensor cores share
// products of 256 rows: each CTA holds half of the keys and half of the value
// components of a tile, so that both the reads and the arrivals halve and three
// stages of 128 keys fit. P is handed over in two parts, so that the products begin
// while the rest of it is made. A pair's tile of keys then takes 2870 cycles, its
// products 2720. Where a pair has 256 rows or fewer, A and B are the same rows and
// take key tiles in turn; their threads join O and the sums at the end.
//
// The grid has a place for every piece (longest sequences first), but a CTA or pair
// that nears the end of its piece takes over one whose place has not started: set-up,
// first loads and epilogue of consecutive pieces then overlap (16 chunks of 300 rows,
// 64 heads, nothing before: 203 -> 141 us; 7 of 1265, 58 heads: 395 -> 294).
//
// Measured, per call in a graph of twelve: four chunks of 2048 rows after 2000 to 16384,
// 16 heads, 735 GFLOP, in 455 us (1.62 PFLOP/s, 82 % of the measured bf16 rate, 94 % of
// the sustained one, which the power limit sets); eight chunks of 512 rows after 0 to
// 8192, 166 GFLOP, in 124 us (68 %: 128 pieces of unequal length over 76 pairs of CTAs,
// of which the longest chains are a fifth longer than the mean). In a long run of single
// calls on changing inputs 490 (76 %) and 130 us (65 %). A softcap costs as much again (the
// special-function units): 228 us for eight chunks of 512 that take 111 without.
#include <math.h>

#include "latent.cuh"

namespace psw {
namespace lpre {

constexpr int kQk = kLatentNope + kLatentRope;
constexpr int kRows = 128;                    // of a row tile
constexpr int kQChunks = kQk / 64;
constexpr int kQUnit = kRows * 128;           // 64 columns of a row tile
constexpr int kQBytes = 2 * kQChunks * kQUnit;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kRoleWarps = 10;
// Three warpgroups (two warps of the last have no role), so that registers can be
// moved: of the 168 a thread that 384 are launched with, a pair's softmax threads, with
// 128 scores each, take 200 (466 -> 458 us for four chunks of 2048 rows; single CTAs,
// with 96, are faster without: 126 against 128 us for 16 chunks of 128).
constexpr int kThreads = 384, kSoftRegs = 200, kOtherRegs = 104;
static_assert(2 * kSoftRegs + kOtherRegs <= 3 * 168, "registers launched with");
constexpr int kTmemS = 0, kTmemO = 256;       // + 128 for B
constexpr float kLag = 64.f;
constexpr int kRanked = 256;                  // sequences put in order by their length
constexpr int kMaxStages = 3;
constexpr int kMisc = 5120;
constexpr int kHead = 64;                     // keys whose P is handed over first

template <int CTAS>
struct Cfg {
  static constexpr int kKeys = CTAS == 2 ? 128 : 96;         // of a key tile
  static constexpr int kStages = CTAS == 2 ? 3 : 2;
  static constexpr int kHeld = kKeys / CTAS;                 // keys that a CTA holds
  static constexpr int kKeyUnit = kHeld * 128;               // 64 columns of them
  static constexpr int kKeyBytes = 3 * kKeyUnit;             // nope, nope, rope
  static constexpr int kValueUnits = 2 / CTAS;               // 64 components each
  static constexpr int kValueUnit = kKeys * 128;
  static constexpr int kValueBytes = kValueUnits * kValueUnit;
  static constexpr int kSmemBytes = 1024 + kQBytes + kStages * (kKeyBytes + kValueBytes) + kMisc;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
};

struct Misc {
  // (the first CTA of a pair: its own and the second's)
  uint64_t k_full[kMaxStages], v_full[kMaxStages], q_full[2];
  uint64_t v_fix[kMaxStages];  // where a value tile with hidden rows lands first
  uint64_t freed[kMaxStages];  // keys of tile k (and values of tile k - 1) are done with
  uint64_t q_free[2];          // the queries of a piece are done with
  uint64_t s_full[2], o_full[2];
  uint64_t p_head[2], p_full[2];  // P of the first kHead keys, of all
  uint64_t drained;
  uint64_t next_full[2], next_empty[2];  // the next piece of work, pieces in turn
  uint4 next[2];
  uint32_t tmem;
  int32_t abort;
  int32_t len[kRanked], order[kRanked];  // sequences, longest first
  float2 ml[2][kRows];   // split: maximum and sum of each row over A's and over B's tiles
};
static_assert(sizeof(Misc) <= kMisc, "misc block");

// A sequence's rows and keys, and what a block of rows has of them; the same in
// every thread.
struct Seq {
  int q0, nq, k0, nk;   // first row and rows (of q), first key row and keys
  int64_t past, first;  // positions of the first row and of the first key
};
struct Work {
  int lo[2], hi[2];     // key tiles [lo, hi) of A and of B
  int t_lo, t_hi;       // of both
  int j_lo, j_hi;       // keys [j_lo, j_hi) that some row sees
};
// Of the rows from i0 on, `tile` in each of A and B, and key tiles of `keys`. Split:
// the same rows in both, every second key tile from lo on.
__device__ __forceinline__ Work work_of(const Seq& q, int i0, int tile, int keys, int window,
                                        bool split) {
  Work w;
  w.t_lo = w.j_lo = 0x7fffffff;
  w.t_hi = w.j_hi = 0;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    if (g == 1 && split) {
      w.lo[1] = w.lo[0] + 1;
      w.hi[1] = w.hi[0];
      break;
    }
    const int n = min(tile, q.nq - i0 - g * tile);
    // keys of the tile's rows: from the window of its first to its last
    const int64_t a = q.past + i0 + g * tile - q.first;
    const int64_t lo64 = window > 0 ? a - window + 1 : 0;
    const int lo = static_cast<int>(max(min(lo64, static_cast<int64_t>(q.nk)), static_cast<int64_t>(0)));
    const int hi = static_cast<int>(max(min(a + n, static_cast<int64_t>(q.nk)), static_cast<int64_t>(0)));
    const bool some = n > 0 && lo < hi;
    w.lo[g] = some ? lo / keys : 0;
    w.hi[g] = some ? (hi + keys - 1) / keys : 0;
    if (some) {
      w.t_lo = min(w.t_lo, w.lo[g]);
      w.t_hi = max(w.t_hi, w.hi[g]);
      w.j_lo = min(w.j_lo, lo);
      w.j_hi = max(w.j_hi, hi);
    }
  }
  return w;
}

template <int CTAS, bool SPLIT, bool FAR_CAP>
__global__ void __launch_bounds__(kThreads, 1)
latent_prefill_kernel(const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap kv_map,
                      const __grid_constant__ CUtensorMap rope_map,
                      const int32_t* __restrict__ cu_q, const int32_t* __restrict__ past_lens,
                      int n_seqs, int n_q, int max_q_len, const int32_t* __restrict__ cu_k,
                      const int32_t* __restrict__ k_first, int n_k, int heads, int blocks,
                      int window, float scale, float softcap, __nv_bfloat16* __restrict__ out,
                      float* __restrict__ lse, int32_t* err) {
  using C = Cfg<CTAS>;
  constexpr int kKeys = C::kKeys, kStages = C::kStages;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* q_smem = smem;
  uint8_t* k_smem = smem + kQBytes;
  uint8_t* v_smem = k_smem + kStages * C::kKeyBytes;
  Misc* ms = reinterpret_cast<Misc*>(v_smem + kStages * C::kValueBytes);

  const int peer = CTAS == 2 ? static_cast<int>(lat::cluster_rank()) : 0;  // number in the pair
  constexpr int kTile = kRows * CTAS;  // rows of A (and of B), of both CTAs
  if (warp == kMmaWarp) {
    if (CTAS == 2) {
      lat::alloc_pair(&ms->tmem, 512);
    } else {
      tc::alloc(&ms->tmem, 512);
      tc::relinquish();
    }
  }
  if (tid == 32 * kLoadWarp) {
    const uint32_t arrivals = CTAS - peer;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&ms->k_full[i], arrivals);
      mbar_init(&ms->v_full[i], arrivals);
      mbar_init(&ms->v_fix[i], 1);
      mbar_init(&ms->freed[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms->q_full[i], arrivals);
      mbar_init(&ms->q_free[i], 1);
      mbar_init(&ms->s_full[i], 1);
      mbar_init(&ms->p_head[i], 4 * CTAS);
      mbar_init(&ms->p_full[i], 4 * CTAS);
      mbar_init(&ms->o_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms->next_full[i], 1);
      mbar_init(&ms->next_empty[i], kRoleWarps * CTAS);
    }
    mbar_init(&ms->drained, 1);
    ms->abort = 0;
    fence_mbar_init();
  }
  // sequences by the work of their last row, ties by index
  if (n_seqs <= kRanked) {
    for (int b = tid; b < n_seqs; b += kThreads) ms->len[b] = __ldg(cu_k + b + 1) - __ldg(cu_k + b);
    __syncthreads();
    for (int b = tid; b < n_seqs; b += kThreads) {
      int ahead = 0;
      const int mine = ms->len[b];
      for (int o = 0; o < n_seqs; ++o) ahead += ms->len[o] > mine || (ms->len[o] == mine && o < b);
      ms->order[ahead] = b;
    }
  }
  __syncwarp();
  tc::fence_before();
  if (CTAS == 2) lat::cluster_sync();
  else __syncthreads();
  tc::fence_after();
  const uint32_t tmem = ms->tmem;
  volatile int32_t* abort_flag = &ms->abort;
  bool ok = true;

  // ---- a piece of work: sequence, head and block of rows. Heads are innermost within
  // a sequence's blocks, its last block (the most keys) first. A CTA's or pair's first
  // piece is that of its place in the grid; the others are those of places that have not
  // started when it asks.
  struct Piece {
    int head, i0, my_row;  // first row of A, of this CTA's part of it
    Seq sq;
    Work w;
  };
  constexpr int b_rows = SPLIT ? 0 : kTile;  // how much further B's rows are
  constexpr int step = SPLIT ? 2 : 1;        // from a key tile of A (or B) to the next
  auto piece_of = [&](int place) {
    Piece x;
    const int item = place / CTAS, per_seq = heads * blocks;
    const int rank = item / per_seq, sub = item - rank * per_seq;
    const int block = blocks - 1 - sub / heads;
    x.head = sub % heads;
    x.i0 = block * 2 * kTile;
    x.my_row = x.i0 + peer * kRows;
    const int b = n_seqs <= kRanked ? ms->order[rank] : rank;
    Seq& sq = x.sq;
    sq.q0 = __ldg(cu_q + b);
    sq.k0 = __ldg(cu_k + b);
    sq.nq = __ldg(cu_q + b + 1) - sq.q0;
    sq.nk = __ldg(cu_k + b + 1) - sq.k0;
    sq.past = __ldg(past_lens + b);
    sq.first = k_first != nullptr ? __ldg(k_first + b) : 0;
    bool bad = false;
    if (sq.q0 < 0 || sq.nq < 0 || sq.past < 0 || sq.k0 < 0 || sq.nk < 0 || sq.first < 0) {
      bad = true;
      sq.nq = sq.nk = 0;
    }
    if (sq.nq > max_q_len || static_cast<int64_t>(sq.q0) + sq.nq > n_q) {
      bad = true;
      sq.nq = max(0, min(sq.nq, min(max_q_len, n_q - sq.q0)));
    }
    if (static_cast<int64_t>(sq.k0) + sq.nk > n_k) {
      bad = true;
      sq.nk = max(0, min(sq.nk, n_k - sq.k0));
    }
    if (bad && tid == 0 && block == 0 && x.head == 0) flag_error(err, PSW_DEVERR_LENGTH);
    x.w = work_of(sq, x.i0, kTile, kKeys, window, SPLIT);
    return x;
  };
  // place of the piece after number `it`, or -1 (called once by every warp)
  auto next_place = [&](int it) {
    if (SPLIT) return -1;  // (there are no more pieces than pairs that run at once)
    ok = __all_sync(0xffffffffu, ok && mbar_wait(&ms->next_full[it & 1], it >> 1 & 1));
    if (!ok) return -1;
    const int place = lat::work_given(&ms->next[it & 1]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (CTAS == 2) lat::arrive_at_first(&ms->next_empty[it & 1]);
      else mbar_arrive(&ms->next_empty[it & 1]);
    }
    return place;
  };

  if (warp >= kLoadWarp) {
    if (CTAS == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      // ------------------------------------------------------------ loads
      const bool one = lat::elect_one();
      uint32_t fixes = 0;      // phases of v_fix
      int n = 0;               // key tiles loaded
      int loaded[2] = {0, 0};  // times that queries of A and of B were loaded
      int asked = -1;          // number of the last piece that the next was asked for in
      for (int place = blockIdx.x, it = 0; ok && place >= 0; ++it) {
        const Piece x = piece_of(place);
        const Work& w = x.w;
        for (int j = w.t_lo; ok && j < w.t_hi; ++j, ++n) {
          const int row = x.sq.k0 + j * kKeys, st = n % kStages;
          auto freed = [&](int k) {  // keys of tile k, values of the one before
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&ms->freed[k % kStages], k / kStages & 1u) && *abort_flag == 0);
            return ok;
          };
          if (n == kStages && !freed(0)) break;  // (later keys: known from the values before them)
          if (one) {  // a pair: half of the keys each
            const uint32_t k = smem_u32(k_smem + st * C::kKeyBytes);
            const int mine = row + peer * C::kHeld;
            mbar_arrive_expect_tx(&ms->k_full[st], C::kKeyBytes);
            lat::tma_box(k, &kv_map, &ms->k_full[st], 0, x.head, mine);
            lat::tma_box(k + C::kKeyUnit, &kv_map, &ms->k_full[st], 64, x.head, mine);
            lat::tma_box(k + 2 * C::kKeyUnit, &rope_map, &ms->k_full[st], 0, mine, 0);
          }
          if (j == w.t_lo) {
            // queries, when those of the piece before are done with
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              if (w.lo[g] >= w.hi[g]) continue;
              if (loaded[g] > 0)
                ok = ok && __all_sync(0xffffffffu, mbar_wait(&ms->q_free[g], (loaded[g] - 1) & 1));
              if (!ok) break;
              ++loaded[g];
              if (one) {
                mbar_arrive_expect_tx(&ms->q_full[g], kQChunks * kQUnit);
                for (int c = 0; c < kQChunks; ++c)
                  lat::tma_box(smem_u32(q_smem + (g * kQChunks + c) * kQUnit), &q_map, &ms->q_full[g],
                               c * 64, x.head, x.sq.q0 + x.my_row + g * b_rows);
              }
            }
          }
          // values (a pair: half of the components each); rows of keys that no row sees
          // (other sequences', or anything) must not enter the second product (P is 0
          // there, but 0 times NaN is not)
          if (!ok || (n >= kStages && !freed(n - kStages + 1))) {
            ++n;  // (its keys are on their way)
            break;
          }
          const int z_lo = w.j_lo - j * kKeys, z_hi = w.j_hi - j * kKeys;
          const bool fix = z_lo > 0 || z_hi < kKeys;
          uint8_t* v = v_smem + st * C::kValueBytes;
          if (one) {
            uint64_t* bar = fix ? &ms->v_fix[st] : &ms->v_full[st];
            mbar_arrive_expect_tx(bar, C::kValueBytes);
#pragma unroll
            for (int c = 0; c < C::kValueUnits; ++c)
#pragma unroll
              for (int h = 0; h < CTAS; ++h)  // (boxes are kHeld rows high)
                lat::tma_box(smem_u32(v + c * C::kValueUnit + h * C::kKeyUnit), &kv_map, bar,
                             kLatentNope + (c + peer) * 64, x.head, row + h * C::kHeld);
          }
          __syncwarp();
          if (fix) {
            ok = __all_sync(0xffffffffu, mbar_wait(&ms->v_fix[st], fixes >> st & 1u));
            fixes ^= 1u << st;
            if (!ok) {
              ++n;
              break;
            }
            for (int i = lane; i < C::kValueUnits * kKeys * 8; i += 32) {
              const int r = (i >> 3) % kKeys;
              if (r < z_lo || r >= z_hi) *reinterpret_cast<uint4*>(v + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms->v_full[st]);
          }
        }
        // With this piece's last loads under way, three tiles before its end, the next is
        // asked for (at this one's beginning, long pieces would be handed out too soon: 140
        // us instead of 130 for eight chunks of 512 rows). The answer's place is free when
        // every warp has read the one two pieces ago.
        if (!SPLIT && peer == 0 && it >= 2)
          ok = ok && __all_sync(0xffffffffu, mbar_wait(&ms->next_empty[it & 1], (it >> 1) - 1 & 1));
        if (!ok) break;
        if (!SPLIT && one) {
          mbar_arrive_expect_tx(&ms->next_full[it & 1], 16);
          if (peer == 0) lat::ask_for_work<CTAS == 2>(&ms->next[it & 1], &ms->next_full[it & 1]);
        }
        asked = it;
        place = next_place(it);
      }
      if (!ok && one) {
        *abort_flag = 1;
        flag_error(err, PSW_DEVERR_PIPELINE);
        // copies and the answer in flight land before the CTA ends
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (loaded[g] > 0) mbar_wait(&ms->q_full[g], (loaded[g] - 1) & 1);
        for (int i = max(0, n - kStages); i < n; ++i) {
          mbar_wait(&ms->k_full[i % kStages], i / kStages & 1);
          mbar_wait(&ms->v_full[i % kStages], i / kStages & 1);
        }
        if (!SPLIT && asked >= 0) mbar_wait(&ms->next_full[asked & 1], asked >> 1 & 1);
      }
    } else if (warp == kMmaWarp && peer == 1) {
      // ------------------------------------------------------------ second CTA of a pair
      // tells the first, which issues the products, what has landed here
      const bool one = lat::elect_one();
      auto pass_on = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && mbar_wait(bar, parity & 1u);
        if (ok && one) lat::arrive_at_first(bar);
      };
      int k = 0, loaded[2] = {0, 0};
      for (int place = blockIdx.x, it = 0; ok && place >= 0; place = next_place(it), ++it) {
        const Work w = piece_of(place).w;
        if (w.t_lo >= w.t_hi) continue;
        pass_on(&ms->k_full[k % kStages], k / kStages);
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (w.lo[g] < w.hi[g]) pass_on(&ms->q_full[g], loaded[g]++);
        for (int j = w.t_lo; ok && j < w.t_hi; ++j, ++k) {
          if (j > w.t_lo) pass_on(&ms->k_full[k % kStages], k / kStages);
          pass_on(&ms->v_full[k % kStages], k / kStages);
        }
      }
      if (one) {
        if (!ok) {
          *abort_flag = 1;
          flag_error(err, PSW_DEVERR_PIPELINE);
        }
        mbar_wait(&ms->drained, 0);  // the last of the first CTA's arrivals here
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ MMAs
      const bool one = lat::elect_one();
      constexpr uint32_t id_s = tc::idesc_bf16_f32(kTile, kKeys, 0, 0);
      constexpr uint32_t id_o = tc::idesc_bf16_f32(kTile, kLatentV, 0, 1);
      const uint64_t q_desc = tc::smem_desc(smem_u32(q_smem), 16, 1024, tc::kSwizzle128B);
      const uint64_t k_desc = tc::smem_desc(smem_u32(k_smem), 16, 1024, tc::kSwizzle128B);
      const uint64_t v_desc = tc::smem_desc(smem_u32(v_smem), C::kValueUnit, 1024, tc::kSwizzle128B);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && mbar_wait(bar, parity & 1u);
      };
      auto commit = [&](uint64_t* bar) {
        if (CTAS == 2) lat::commit_pair(bar);
        else tc::commit(bar);
      };
      int n[2] = {0, 0};       // S formed for each row tile
      int loaded[2] = {0, 0};  // and times that its queries were waited for
      bool fresh[2] = {};      // none in this piece so far
      auto scores = [&](int g, int k, bool last) {  // of the k-th key tile loaded, this piece's last
        if (fresh[g]) wait(&ms->q_full[g], loaded[g]++);
        fresh[g] = false;
        tc::fence_after();
        const uint64_t kd = k_desc + (k % kStages) * (C::kKeyBytes >> 4);
        const uint64_t qd = q_desc + g * kQChunks * (kQUnit >> 4);
        if (ok && one) {
#pragma unroll
          for (int c = 0; c < kQChunks; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint64_t a = qd + (c * kQUnit >> 4) + e * 2, b = kd + (c * C::kKeyUnit >> 4) + e * 2;
              const uint32_t acc = (c > 0 || e > 0) ? 1u : 0u;
              if (CTAS == 2) lat::mma_ss_pair(tmem + kTmemS + g * 128, a, b, id_s, acc);
              else tc::mma_ss(tmem + kTmemS + g * 128, a, b, id_s, acc);
            }
          commit(&ms->s_full[g]);
          if (last) commit(&ms->q_free[g]);
        }
        ++n[g];
      };
      // the k-th key tile has landed, the k-th value tile has
      auto keys = [&](int k) { wait(&ms->k_full[k % kStages], k / kStages); };
      auto values = [&](int k) { wait(&ms->v_full[k % kStages], k / kStages); };
      int k = 0;  // key tiles so far
      for (int place = blockIdx.x, it = 0; ok && place >= 0; place = next_place(it), ++it) {
        const Work w = piece_of(place).w;
        if (w.t_lo >= w.t_hi) continue;
        auto has = [&](int g, int j) {
          return j >= w.lo[g] && j < w.hi[g] && (!SPLIT || ((j ^ w.lo[g]) & 1) == 0);
        };
        fresh[0] = fresh[1] = true;
        keys(k);
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (w.lo[g] == w.t_lo && w.lo[g] < w.hi[g]) scores(g, k, w.lo[g] + step >= w.hi[g]);
        if (ok && one) commit(&ms->freed[k % kStages]);
        values(k);
        if (w.t_lo + 1 < w.t_hi) {
          keys(k + 1);
          if (SPLIT) scores(1, k + 1, w.lo[1] + step >= w.hi[1]);
        }
        for (int j = w.t_lo; ok && j < w.t_hi; ++j, ++k) {
          const int st = k % kStages;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (has(g, j)) {
              const uint64_t vd = v_desc + st * (C::kValueBytes >> 4);
              auto product = [&](int e) {
                const uint32_t d = tmem + kTmemO + g * kLatentV, a = tmem + kTmemS + g * 128 + e * 8;
                const uint32_t acc = (j > w.lo[g] || e > 0) ? 1u : 0u;
                if (CTAS == 2) lat::mma_ts_pair(d, a, vd + e * (2048 >> 4), id_o, acc);
                else tc::mma_ts(d, a, vd + e * (2048 >> 4), id_o, acc);
              };
              wait(&ms->p_head[g], n[g] - 1);
              tc::fence_after();
              if (ok && one) {
#pragma unroll
                for (int e = 0; e < kHead / 16; ++e) product(e);
              }
              wait(&ms->p_full[g], n[g] - 1);
              tc::fence_after();
              if (ok && one) {
#pragma unroll
                for (int e = kHead / 16; e < kKeys / 16; ++e) product(e);
                if (j + step >= w.hi[g]) commit(&ms->o_full[g]);
              }
            }
            if (SPLIT) {
              if (has(g, j) && j + 2 < w.hi[g]) {
                keys(k + 2);
                scores(g, k + 2, j + 2 + step >= w.hi[g]);
              }
            } else if (has(g, j + 1)) {
              scores(g, k + 1, j + 1 + step >= w.hi[g]);
            }
            if (g == 0) {  // what the next round needs, while B's softmax runs
              if (j + 1 < w.t_hi) values(k + 1);
              if (j + 2 < w.t_hi) keys(k + 2);
            }
          }
          if (ok && one && j + 1 < w.t_hi) commit(&ms->freed[(k + 1) % kStages]);
        }
      }
      if (one) {
        if (!ok) {
          *abort_flag = 1;
          flag_error(err, PSW_DEVERR_PIPELINE);
        }
        commit(&ms->drained);  // every product has ended before tensor memory is freed
        mbar_wait(&ms->drained, 0);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax, epilogue
    if (CTAS == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int g = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + kTmemS + g * 128;
    const uint32_t o_at = tmem + lanes + kTmemO + g * kLatentV;
    const bool cap = softcap > 0.f;
    const float mul = cap ? 1.f : scale * lat::kLog2e;
    const float cap_in = cap ? scale / softcap : 0.f, cap_out = softcap * lat::kLog2e;
    int formed = 0;             // S so far
    uint32_t ends = 0;          // phases of o_full
    // what this thread has of a piece: its row's visible keys [first, last], its half's key
    // tiles, and where its results go (row -1: nowhere)
    struct Mine {
      int first, last, lo, hi;
      bool other;  // split: the other half has key tiles
      int64_t row;
    };
    auto mine_of = [&](int place) {
      const Piece x = piece_of(place);
      const int i = x.my_row + g * b_rows + r;
      const int64_t p = x.sq.past + i - x.sq.first;  // relative to the first key
      Mine y;
      y.last = static_cast<int>(max(min(p, static_cast<int64_t>(x.sq.nk - 1)), static_cast<int64_t>(-1)));
      y.first = window > 0 ? static_cast<int>(max(min(p - window + 1, static_cast<int64_t>(x.sq.nk)),
                                                  static_cast<int64_t>(0)))
                           : 0;
      y.lo = g == 0 ? x.w.lo[0] : x.w.lo[1];
      y.hi = g == 0 ? x.w.hi[0] : x.w.hi[1];
      y.other = SPLIT && (g == 0 ? x.w.lo[1] < x.w.hi[1] : x.w.lo[0] < x.w.hi[0]);
      y.row = i < x.sq.nq ? static_cast<int64_t>(x.sq.q0 + i) * heads + x.head : -1;
      return y;
    };
    Mine x = mine_of(blockIdx.x);
    for (int it = 0; ok; ++it) {
      float m = -INFINITY, l = 0.f;
      for (int j = x.lo; j < x.hi; j += step, ++formed) {
        // (every decision is the same in the whole warp)
        ok = __all_sync(0xffffffffu, mbar_wait(&ms->s_full[g], formed & 1) && *abort_flag == 0);
        if (!ok) break;
        tc::fence_after();
        float z[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys / 32; ++c)
          tc::ld32(s_at + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&z[c * 32]));
        tc::wait_ld();
        // this row's visible columns of the tile
        const int c_hi = min(x.last - j * kKeys, kKeys - 1), c_lo = max(x.first - j * kKeys, 0);
        if (cap) {
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            z[c] = cap_out * (FAR_CAP ? lat::tanh_of(z[c] * cap_in) : lat::tanh_large(z[c] * cap_in));
        }
        if (!__all_sync(0xffffffffu, c_lo <= 0 && c_hi >= kKeys - 1)) {
#pragma unroll
          for (int c = 0; c < kKeys; ++c) z[c] = c >= c_lo && c <= c_hi ? z[c] : -INFINITY;
        }
        float mx[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
        for (int c = 4; c < kKeys; c += 8) {
          mx[0] = max3f(mx[0], z[c], z[c + 1]);
          mx[1] = max3f(mx[1], z[c + 2], z[c + 3]);
          if (c + 4 < kKeys) {
            mx[2] = max3f(mx[2], z[c + 4], z[c + 5]);
            mx[3] = max3f(mx[3], z[c + 6], z[c + 7]);
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
            // (the product of the tile before was issued before this S, and has ended)
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
        uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < kKeys / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 d = f2_unpack(f2_fma(f2_pack(z[c * 32 + 2 * e], z[c * 32 + 2 * e + 1]), mul2, ref2));
            const float a0 = ex2_approx(d.x), a1 = ex2_approx(d.y);
            sum[e & 1] = f2_add(sum[e & 1], f2_pack(a0, a1));
            pk[e] = pack_bf16x2(a0, a1);
          }
          tc::st16(s_at + c * 16, pk);
          if (c * 32 + 32 == kHead || c * 32 + 32 == kKeys) {
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            uint64_t* bar = c * 32 + 32 == kHead ? &ms->p_head[g] : &ms->p_full[g];
            if (lane == 0) {
              if (CTAS == 2) lat::arrive_at_first(bar);
              else mbar_arrive(bar);
            }
          }
        }
        const float2 sums0 = f2_unpack(sum[0]), sums1 = f2_unpack(sum[1]);
        l += (sums0.x + sums0.y) + (sums1.x + sums1.y);
      }
      // (the piece after this one, looked up while the last products run)
      const int place = ok ? next_place(it) : -1;
      const bool some = x.lo < x.hi, other = x.other, mine = x.row >= 0;
      const int64_t row = x.row;
      if (place >= 0) x = mine_of(place);
      if (some) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&ms->o_full[g], ends >> g & 1u));
        ends ^= 1u << g;
      }
      uint4* dst = reinterpret_cast<uint4*>(out + row * kLatentV);
      if constexpr (SPLIT) {
        // A's threads and B's have the same rows, each the sums over its own key tiles;
        // they join them, 64 components each (a lane's O is there for both)
        ms->ml[g][r] = make_float2(m, l);
        named_bar_sync(1, 256);
        const float2 o = ms->ml[1 - g][r];
        const float top = fmaxf(m, o.x);
        float f = m == -INFINITY ? 0.f : ex2_approx(m - top);
        float f_other = o.x == -INFINITY ? 0.f : ex2_approx(o.x - top);
        l = l * f + o.y * f_other;
        m = top;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        f *= inv;
        f_other *= inv;
        if (other) {
          ok = ok && __all_sync(0xffffffffu, mbar_wait(&ms->o_full[1 - g], ends >> (1 - g) & 1u));
          ends ^= 1u << (1 - g);
        }
        if (ok) {
          tc::fence_after();
          const uint32_t o_other = tmem + lanes + kTmemO + (1 - g) * kLatentV;
#pragma unroll 1
          for (int c = 2 * g; c < 2 * g + 2; ++c) {
            uint32_t v[32], u[32];
            if (some) tc::ld32(o_at + c * 32, v);
            if (other) tc::ld32(o_other + c * 32, u);
            tc::wait_ld();
            if (!mine) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float y[8];
#pragma unroll
              for (int d = 0; d < 8; ++d) {
                y[d] = f == 0.f ? 0.f : __uint_as_float(v[e * 8 + d]) * f;
                if (f_other != 0.f) y[d] = fmaf(__uint_as_float(u[e * 8 + d]), f_other, y[d]);
              }
              dst[c * 4 + e] = lat::pack8(y);
            }
          }
        }
      } else if (ok) {
        tc::fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          if (some) {
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
      }
      if (ok && mine && lse != nullptr && (g == 0 || !SPLIT))
        lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * lat::kLn2;
      // O has been read before the P of the next piece lets it be written (split: by
      // the threads of both)
      tc::fence_before();
      if (SPLIT && lat::bar_any(1, 256, !ok)) ok = false;
      if (place < 0) break;
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      flag_error(err, PSW_DEVERR_PIPELINE);
    }
  }
  __syncwarp();
  tc::fence_before();
  if (CTAS == 2) lat::cluster_sync();  // nobody leaves while the other may still reach into it
  else __syncthreads();
  if (warp == kMmaWarp) {
    if (CTAS == 2) lat::dealloc_pair(tmem, 512);
    else tc::dealloc(tmem, 512);
  }
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
  max_q_len = min(max_q_len, n_q_total);  // (no chunk within the rows is longer)
  // Pairs of CTAs for chunks that are longer than the 256 rows of one (8 chunks of 384
  // rows after 4096, 16 heads: 131 us against 155), and where all pairs run at once:
  // shorter ones then have their keys split between A and B (1 of 256 after 8192, 76
  // heads: 84 us against 173; 4 of 128 after 8192, 16 heads: 79 against 111). With more
  // work than that SMs are what is short (16 of 128 after 4096, 16 heads: 173 against
  // 134). Single CTAs do not split: their two stages hold no tile ahead of the two in
  // use (the same: 180).
  const bool spare = 2 * static_cast<int64_t>(n_seqs) * L.n_heads <= num_sms;
  const int ctas = max_q_len > 2 * kRows || spare ? 2 : 1;
  const bool split = ctas == 2 && max_q_len <= kRows * ctas;
  const int held = ctas == 2 ? Cfg<2>::kHeld : Cfg<1>::kHeld;
  const int64_t blocks = (static_cast<int64_t>(max_q_len) + 2 * kRows * ctas - 1) / (2 * kRows * ctas);
  const int64_t grid = blocks * ctas * L.n_heads * n_seqs;
  if (grid > 0x7fffffffLL) return PSW_ECAPACITY;
  int rc = make_map_3d(&q_map, false, q, {kQk, h, n_q_total}, {2 * kQk, 2 * kQk * h}, {64, 1, kRows});
  if (rc != PSW_OK) return rc;
  if (n_k_total > 0) {
    rc = make_map_3d(&kv_map, false, kv, {kLatentKv, h, n_k_total}, {2 * kLatentKv, 2 * kLatentKv * h},
                     {64, 1, held});
    if (rc == PSW_OK)
      rc = make_map_3d(&rope_map, false, k_rope, {kLatentRope, n_k_total, 1},
                       {2 * kLatentRope, 2 * kLatentRope}, {64, held, 1});
    if (rc != PSW_OK) return rc;
  } else {
    kv_map = rope_map = q_map;  // no key tile will be loaded
  }
  // (as a run-time choice the form for large caps cost the others 3 to 10 %)
  const bool far = L.softcap > lat::kNearCap;
  auto* kernel = split       ? (far ? latent_prefill_kernel<2, true, true> : latent_prefill_kernel<2, true, false>)
                 : ctas == 2 ? (far ? latent_prefill_kernel<2, false, true> : latent_prefill_kernel<2, false, false>)
                             : (far ? latent_prefill_kernel<1, false, true> : latent_prefill_kernel<1, false, false>);
  const int smem = ctas == 2 ? Cfg<2>::kSmemBytes : Cfg<1>::kSmemBytes;
  rc = set_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  if (rc != PSW_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, kernel, q_map, kv_map, rope_map, cu_q, past_lens, n_seqs, n_q_total, max_q_len, cu_k,
      k_first, n_k_total, L.n_heads, static_cast<int>(blocks), L.window, L.scale, L.softcap,
      static_cast<__nv_bfloat16*>(out), lse, err);
  return e == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

}  // namespace psw
