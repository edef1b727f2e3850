// latent_decode.cu -- absorbed latent attention of one token per sequence over
// its pages (split along the context, joined by the log-sum-exp rule).
//
// Mathematics, per sequence and head over the visible rows j:
//   s_j = softcap(scale <q, row_j>),  out = sum_j softmax(s)_j row_j[:L].
// Each cached row is read once for all heads (a chunk of up to 32), so the
// call is bound by HBM: 2 (2 L + 64) operations a byte pair and head, 60 a byte
// at 32 heads. That is far beyond what the CUDA cores and more than what
// mma.sync sustain beside the loads, so both products run on tcgen05, turned
// so that the padded operand side is the large one:
//   S^T [64 keys x heads]   = K Q^T      (A: key rows as stored, K-major)
//   O^T [128 dims x heads] += V^T P^T    (A: the same rows, read MN-major)
// with the heads as the N side (16 or 32) and no wasted rows.
//
// Precision. bf16 pages: P enters as a bf16 part and the bf16 of the rest, two
// column groups of one N (the A side is read once for both; one part alone
// would add as much error as the output's own rounding). FP8 pages: the codes
// are A as they are. q, times a power of two, is the sum of two E4M3 parts (all 8
// bits of a value, but for 2^-21 of the head's largest). A row's weight, P times its
// scale, is taken in three parts, each 16 times finer than the one before: off by 2^-12
// of itself, or by 2^-18 units where the third is subnormal. A head's unit is a power
// of two, chosen so that the largest weight of a tile is 8 units, and chosen anew (O
// rescaled) at a tile whose largest is beyond the codes, or below 2^-4 while 2^-18 units
// of each of the segment's rows could add up to more than 2^-9 of the probability: rows
// that follow one of large score or scale weigh little beside it, but there may be
// many. (Where the rows' scales are alike that is so of segments of 2000 rows or more;
// always when it is below 2^-4: 45 us instead of 37 for 64 sequences whose scores have
// a deviation of 2.9.) What a tile's 64 rows are off by is thus 2^-12 + 2^-8 of their
// sum at worst, or at most 2^-9 of the probability in all. Row scales multiply scores
// and P in fp32. Maxima and sums are fp32.
//
// Schedule: one CTA per SM. The visible pages of all (sequence, head chunk)
// units form one list that is cut evenly; a CTA whose piece covers a unit
// writes the result, the others leave (O, m, l) for latent_merge_kernel. Tiles
// of 64 keys go through a ring of 8 KB slots (64 rows x 128 B, swizzled): a
// tile is its rope unit and L / 128 blocks of 128 dims. L2 feeds an SM no
// faster than HBM does, so the loads must never pause: what counts is how long
// a byte stays in the ring. Hence small tiles (128 keys: slower in every case),
// S of the next tiles ahead of the second product of this one (two buffers of
// S; a warp issues S, another O), MMAs issued from converged code (40 cycles
// each, what reading their operands takes, against 80 to 260), and blocks
// released one by one. The rope slot of a tile is done with after S, and then
// holds P. Four warps for every 16 heads do the softmax (a thread has two keys
// and four heads) and the epilogue (a thread per dim); one warp loads pages,
// one (FP8, which splits them into parts: four) the queries. The maximum that P
// is relative to is taken from a segment's first tile and moved (O rescaled)
// only when a score exceeds it by 2^64 (FP8: wherever units move), so that most tiles
// cost their threads one barrier.
//
// Measured (latent 512, GPU time of a call in a graph of twelve, joins included; single
// calls that follow on one another take the same). 64 sequences of 512 to 4096 rows, 16
// heads: bf16 171 MB in 39.5 us (4.3 TB/s; a kernel that only gathers the pages takes
// 30), FP8 86 MB in 31 us. 32 sequences of 1024 to 32768 rows, 32 heads, bf16: 321 MB
// in 67.5 us (4.8 TB/s). 3 sequences of 40001 to 65536 rows, 24 heads, FP8: 80 MB in 36
// us. About 4 us are start-up (lengths, the cut, the first block ids and pages: loads
// that follow on one another) and 4 the join. In between bf16 is bound by the loads;
// FP8 by a tile's chain (scores, softmax, three parts of P) and, at more than 16 heads,
// by shared memory, from which two parts of q and three of P are read. Heads beyond 32
// are further units, each of which reads its pages again.
#include <math.h>

#include "latent.cuh"

namespace psw {
namespace ldec {

constexpr int kTile = 64;                       // keys of a tile
constexpr int kPages = kTile / kBlockSize;      // pages of a tile
constexpr int kSlotBytes = kTile * 128;
constexpr int kMaxCtas = 160;                   // pieces of the page list
constexpr int kMinPages = 4;                    // pages a piece has at least
constexpr int kMaxHeads = 32;                   // heads of a chunk
constexpr int kSmemLimit = 232448;
// FP8: up to so many heads whose O is rescaled are so column by column, and nothing of
// the others is touched (3 long sequences: 48.7 -> 45.0 us for scores of a deviation of
// 2.9, 39.0 -> 38.1 of 1.7); more go through all columns, as on bf16 pages, where a
// maximum hardly ever moves.
constexpr int kFewHeads = 4;

__host__ __device__ inline int chunk_heads(int heads) { return heads <= 16 ? 16 : 32; }
__host__ __device__ inline int chunks_of(int heads) {
  return (heads + chunk_heads(heads) - 1) / chunk_heads(heads);
}

template <int LAT, int NH, bool FP8>
struct Cfg {
  static constexpr int kElems = FP8 ? 128 : 64;        // row values of a 128-byte slot row
  static constexpr int kBlocks = LAT / 128;            // 128-dim blocks of the latent
  static constexpr int kSlotsPerBlock = 128 / kElems;
  static constexpr int kQParts = FP8 ? 2 : 1, kPParts = FP8 ? 3 : 2;
  static constexpr int kQRows = NH * kQParts;          // N of S^T
  static constexpr int kPCols = NH * kPParts;          // N of O^T
  static constexpr int kQChunks = LAT / kElems + 1;    // 128-byte columns of Q, rope last
  static constexpr int kQChunkBytes = kQRows * 128;
  static constexpr int kQBytes = kQChunks * kQChunkBytes;
  static constexpr int kRopeSteps = FP8 ? 2 : 4;       // 32-byte MMA steps of the rope chunk
  static constexpr int kPSteps = FP8 ? 2 : 4;          // MMA steps along the keys
  static constexpr int kPStepBytes = kTile / kPSteps * 128;
  // Roles by warp: softmax, four warps for every 16 heads; MMAs of S; MMAs of O;
  // pages; queries.
  static constexpr int kGroups = NH / 16;
  static constexpr int kSoftThreads = 128 * kGroups;
  static constexpr int kScoreWarp = 4 * kGroups, kValueWarp = kScoreWarp + 1;
  static constexpr int kLoadWarp = kScoreWarp + 2, kQueryWarp = kScoreWarp + 3;
  static constexpr int kQueryWarps = FP8 ? 4 : 1;
  static constexpr int kThreads = 32 * (kQueryWarp + kQueryWarps);
  static constexpr int kMisc = FP8 ? 6144 : 2560;
  static constexpr int kTileSlots = 1 + kBlocks * kSlotsPerBlock;
  static constexpr int kSlots = (kSmemLimit - 1024 - kMisc - kQBytes) / kSlotBytes;
  static constexpr int kSmemBytes = 1024 + kQBytes + kSlots * kSlotBytes + kMisc;
  static constexpr int kTmemO = 2 * kQRows;            // after the two S^T buffers
  static_assert(kTmemO + kBlocks * kPCols <= 512, "tensor memory columns");
  static_assert(kSlots >= 2 * kTileSlots + 1, "two tiles fit, a slot left out included");
  // FP8: row scales of the tiles in the ring, in turn (after the misc block)
  static constexpr int kScaleTiles = 14;
  static constexpr int kScales = 2560, kScaleBytes = kTile * 4;
  static_assert(!FP8 || (kScales + kScaleTiles * kScaleBytes <= kMisc &&
                         kSlots / kTileSlots + 2 <= kScaleTiles),
                "no tile's scales are overwritten while it is in the ring");
  // Pages that a unit counts for beyond its own: a piece that goes from one unit to
  // the next writes out, loads queries and fills the pipeline again meanwhile
  // (0, 4, 8, 12, 16, 24: 42.5, 41.0, 40.1, 41.0, 41.0, 42.4 us for 64 sequences of
  // bf16 pages; 34.2, 31.8, 31.4, 30.8, 31.4, 33.0 us of FP8 pages).
  static constexpr int kBegin = FP8 ? 12 : 8;
  static constexpr int kHeads = 4;                     // heads of a softmax thread
  static_assert(kSlots <= 32, "phase bits");
  // log2 distance by which a score may exceed the maximum in use
  static constexpr float kLag = 64.f;
  // FP8, log2 of a row's weight in units: the largest of a tile may be at most kMost (448
  // is the largest code), and is kAim where the unit is chosen (3: 4 and 5 moved it more
  // often). It is chosen anew too where the largest is below kLeast and the unit is
  // coarse for some row of the tile: 2^-18 units of every row of the segment, with that
  // row's scale, would be more than 2^(kSpare - 18) of the probability. (kSpare 8 is
  // within what alike scales differ by in segments of 1000 rows: 34 us instead of 32.) A
  // head's unit never falls kReach below what its largest weight so far asked for: that
  // one's share of O then still fits fp32, and what is left out is 2^-40 of it.
  static constexpr float kMost = 8.75f, kLeast = -4.f, kAim = 3.f, kSpare = 9.f, kReach = 40.f;
};

// The list, cut into n pieces: of q + 1 for the first r, of q for the others.
struct Cut {
  int q, r;
  __device__ __forceinline__ int first(int i) const { return q * i + min(i, r); }
  __device__ __forceinline__ int piece(int x) const {  // that holds place x
    const int wide = (q + 1) * r;
    return x < wide ? x / (q + 1) : r + (x - wide) / q;
  }
};

struct Misc {
  uint64_t full[32], empty[32];
  uint64_t q_full, q_free, s_full[2], p_full[3], pv_done[3], o_full, o_free, drained;
  int32_t b0, chunk0, at0;   // this CTA's first unit and the place within it
  uint32_t tmem;
  int32_t abort;
  Cut cut;                   // of what all units count for
  int32_t p0, p1;            // this CTA's piece of it
  float red[4][kMaxHeads];
  float heavy[4][kMaxHeads];  // FP8: by row warp, log2 of the largest weights
  // FP8, by warp: a bit for each of its 16 heads, some key of the tile weighs 2^kLeast units
  // or more, and 16 up, the unit is coarse for some key; whether something has to move up
  alignas(16) uint32_t says[8];
  alignas(16) uint32_t up[8];
  float qs[3][kMaxHeads];    // FP8, segments in turn: scale * log2(e) * a unit of q's codes
  float lsum[kMaxHeads];
  float alpha[kMaxHeads];    // factors of a rescale; at a segment's end, the maxima
  float top[kMaxHeads];      // FP8: the largest weight (log2) seen when units were chosen; at a
                             // segment's end, the root of what a unit stands for
};
static_assert(sizeof(Misc) <= 2560, "misc block");

// Row scales of a page that is not there (its codes read as zeros).
__device__ const float4 g_zero_scales[kBlockSize / 4] = {};

// Visible pages of one sequence.
struct Span {
  int len, lo;          // keys [lo, len)
  int first, count;     // pages
  // what a unit of these pages counts for in the list that is cut evenly
  __device__ __forceinline__ int cost(int begin) const { return count > 0 ? begin + count : 0; }
};
__device__ __forceinline__ Span span_of(int raw, int window, int max_blocks) {
  Span s;
  const int64_t cap = static_cast<int64_t>(max_blocks) * kBlockSize;
  s.len = raw < 0 ? 0 : (raw > cap ? static_cast<int>(cap) : raw);
  s.lo = window > 0 && s.len > window ? s.len - window : 0;
  s.first = s.lo / kBlockSize;
  s.count = s.len > 0 ? (s.len - 1) / kBlockSize - s.first + 1 : 0;
  return s;
}

struct Part {  // what a unit's pieces left behind, per unit: pieces [x, y], x < 0: none
  int32_t x, y;
};

// A CTA's segments in order: each role walks them by itself.
struct Walk {
  const int32_t* seq_lens;
  int window, max_blocks, chunks, n_seqs;
  int left;              // of this CTA's piece (pages, `begin` more for each unit)
  int begin;
  int next_b, next_chunk, at;  // unit that comes next, and the place within what it counts for
  int b, chunk;
  Span span;
  int seg_first, seg_count;  // pages of the segment, relative to the span's first
  __device__ __forceinline__ bool next() {
    while (left > 0 && next_b < n_seqs) {
      span = span_of(seq_lens[next_b], window, max_blocks);
      b = next_b;
      chunk = next_chunk;
      const int cost = span.cost(begin);
      const int take = min(cost - at, left);
      // of [at, at + take) the first `begin` are no pages
      seg_first = max(at - begin, 0);
      seg_count = max(at + take - begin, 0) - seg_first;
      left -= take;
      at += take;
      if (at == cost) {
        at = 0;
        if (++next_chunk == chunks) next_chunk = 0, ++next_b;
      }
      if (seg_count > 0) return true;
    }
    return false;
  }
  __device__ __forceinline__ bool whole() const { return seg_first == 0 && seg_count == span.count; }
  __device__ __forceinline__ int tiles() const { return (seg_count + kPages - 1) / kPages; }
};

// Ring slots in the order of use, and each slot's phase (bit s of `parity`:
// that of this use). A block of two slots does not wrap: the last slot is then
// left out, its phase unchanged.
struct Ring {
  int pos = 0;
  uint32_t phase = 0;
  template <int NS>
  __device__ __forceinline__ int take(int n, uint32_t& parity) {
    if (pos + n > NS) pos = 0;
    const int s = pos;
    parity = phase;
    phase ^= ((1u << n) - 1u) << s;
    pos += n;
    if (pos == NS) pos = 0;
    return s;
  }
};

// The kernels of a call are launched while what is ahead of them in the stream
// may still run: nothing of the inputs, the outputs or the workspace is touched
// before this. What they read may thus be written while they are alive, which rules
// out the read-only path (`__ldg`, and inputs marked const __restrict__): loads
// are plain ones here.
__device__ __forceinline__ void wait_for_inputs() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int LAT, int NH, bool FP8, bool FAR_CAP>
__global__ void __launch_bounds__(Cfg<LAT, NH, FP8>::kThreads, 1)
latent_decode_kernel(const __grid_constant__ CUtensorMap q_map,
                     const __grid_constant__ CUtensorMap pool_map, const LatentPages pages,
                     const __nv_bfloat16* q, const int32_t* seq_lens,
                     int n_seqs, int heads, int window, float scale, float softcap,
                     __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
                     Part* __restrict__ parts, float2* __restrict__ part_ml,
                     float* __restrict__ part_o, int32_t* err, int stall_cta, int stall_tile) {
  using C = Cfg<LAT, NH, FP8>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kSoftThreads = C::kSoftThreads, kScoreWarp = C::kScoreWarp;
  constexpr int kValueWarp = C::kValueWarp, kLoadWarp = C::kLoadWarp, kQueryWarp = C::kQueryWarp;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* q_smem = smem;
  uint8_t* ring = smem + C::kQBytes;
  Misc* ms = reinterpret_cast<Misc*>(ring + C::kSlots * kSlotBytes);
  uint8_t* scales = reinterpret_cast<uint8_t*>(ms) + C::kScales;
  const int chunks = chunks_of(heads);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may queue up

  if (warp == kLoadWarp) {
    // ---- set-up and this CTA's piece of the page list, by the warp whose loads
    // everything waits for: it adds up all spans, a run of sequences per lane,
    // and the lane whose run holds the piece's first page finds the unit
    mbar_init(&ms->full[lane], 1);
    mbar_init(&ms->empty[lane], 1);
    if (lane < 3) {
      if (lane < 2) mbar_init(&ms->s_full[lane], 1);
      mbar_init(&ms->p_full[lane], kSoftThreads / 32);
      mbar_init(&ms->pv_done[lane], 1);
    } else if (lane == 3) {
      mbar_init(&ms->q_full, C::kQueryWarps);
      mbar_init(&ms->q_free, 1);
      mbar_init(&ms->o_full, 1);
      mbar_init(&ms->o_free, kSoftThreads / 32);
      mbar_init(&ms->drained, 2);
      ms->abort = 0;
    }
    fence_mbar_init();
    __syncwarp();
    wait_for_inputs();
    const int per = (n_seqs + 31) / 32;
    const int b0 = min(n_seqs, lane * per), b1 = min(n_seqs, b0 + per);
    int mine = 0;  // (the host has seen to it that 32 bits hold the sum)
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
      const int raw = seq_lens[b];
      mine += span_of(raw, window, pages.max_blocks).cost(C::kBegin) * chunks;
      if (blockIdx.x == 0) {
        if (raw < 0) flag_error(err, PSW_DEVERR_LENGTH);
        if (raw > static_cast<int64_t>(pages.max_blocks) * kBlockSize)
          flag_error(err, PSW_DEVERR_CAPACITY);
      }
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    const int pieces = max(1, min(static_cast<int>(gridDim.x), (total + kMinPages - 1) / kMinPages));
    const Cut cut{total / pieces, total % pieces};
    const bool work = static_cast<int>(blockIdx.x) < pieces;
    const int p0 = work ? cut.first(blockIdx.x) : 0, p1 = work ? cut.first(blockIdx.x + 1) : 0;
    if (p0 < p1 && p0 >= incl - mine && p0 < incl) {
      int at = incl - mine;
      for (int b = b0; b < b1; ++b) {
        const int n = span_of(seq_lens[b], window, pages.max_blocks).cost(C::kBegin);
        if (p0 < at + n * chunks) {
          int c = 0;
          for (; p0 >= at + n; at += n) ++c;
          ms->b0 = b;
          ms->chunk0 = c;
          ms->at0 = p0 - at;
          break;
        }
        at += n * chunks;
      }
    }
    if (lane == 0) {
      ms->cut = cut;
      ms->p0 = p0;
      ms->p1 = p1;
    }
    __threadfence_block();
    __syncwarp();
    // goes straight on; the others come to these barriers when they are ready
    asm volatile("bar.arrive 2, %0;" ::"r"(C::kThreads - kSoftThreads) : "memory");
    asm volatile("bar.arrive 4, %0;" ::"r"(kSoftThreads + 32) : "memory");
  } else {
    if (warp == kScoreWarp) {
      tc::alloc(&ms->tmem, 512);
      tc::relinquish();
    }
    if (warp == kValueWarp && lane == 0) {
      prefetch_tensormap(&pool_map);
      prefetch_tensormap(&q_map);
    }
    if (warp <= kScoreWarp) {
      tc::fence_before();
      named_bar_sync(3, kSoftThreads + 32);
      tc::fence_after();
    }
    if (warp >= kScoreWarp) {  // (the softmax warps come to this later)
      wait_for_inputs();
      named_bar_sync(2, C::kThreads - kSoftThreads);
    }
  }
  const uint32_t tmem = warp <= kScoreWarp || warp == kValueWarp ? ms->tmem : 0u;
  volatile int32_t* abort_flag = &ms->abort;
  Walk walk;
  auto begin = [&]() {  // once the piece is known
    walk.seq_lens = seq_lens;
    walk.window = window;
    walk.max_blocks = pages.max_blocks;
    walk.chunks = chunks;
    walk.n_seqs = n_seqs;
    walk.left = ms->p1 - ms->p0;
    walk.next_b = ms->b0;  // (anything, where there is no page)
    walk.next_chunk = ms->chunk0;
    walk.at = ms->at0;
    walk.begin = C::kBegin;
  };
  if (warp >= kScoreWarp) begin();
  Ring rg;
  bool ok = true;
  const float mul = softcap > 0.f ? scale / softcap : scale * lat::kLog2e;  // (times cap2 later)

  if (warp >= kQueryWarp) {
    // ------------------------------------------------------------ queries
    const int h_first = warp - kQueryWarp;
    int seg = 0;
    for (; ok && walk.next(); ++seg) {
      const int h0 = walk.chunk * NH;
      if constexpr (!FP8) {
        // (the previous unit's queries are done with when its last S is)
        if (seg > 0) ok = __all_sync(0xffffffffu, mbar_wait(&ms->q_free, (seg - 1) & 1));
        if (ok && lat::elect_one()) {
          mbar_arrive_expect_tx(&ms->q_full, C::kQBytes);
#pragma unroll
          for (int c = 0; c < C::kQChunks; ++c)
            lat::tma_box(smem_u32(q_smem + c * C::kQChunkBytes), &q_map, &ms->q_full, c * 64, h0,
                         walk.b);
        }
      } else {
        // a warp has every fourth head: its largest value gives the power of two,
        // a value is the sum of two parts, the second 16 times up
        constexpr int kRow = LAT + kLatentRope, kPairs = kRow / 2, kWords = (kPairs + 31) / 32;
        uint32_t raw[NH / 4][kWords];
#pragma unroll
        for (int j = 0; j < NH / 4; ++j) {
          const int h = h0 + h_first + 4 * j;
          const uint32_t* src = reinterpret_cast<const uint32_t*>(
              q + (static_cast<int64_t>(walk.b) * heads + h) * kRow);
#pragma unroll
          for (int i = 0; i < kWords; ++i)
            raw[j][i] = (h < heads && i * 32 + lane < kPairs) ? src[i * 32 + lane] : 0u;
        }
        if (seg > 0) ok = __all_sync(0xffffffffu, mbar_wait(&ms->q_free, (seg - 1) & 1));
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < NH / 4; ++j) {
          const int h = h_first + 4 * j;
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const float2 v = unpack_bf16x2(raw[j][i]);
            amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
          amax = lat::warp_max(amax);
          // 2^k with amax 2^k in [128, 256), from amax's exponent field
          const int ex = static_cast<int>(__float_as_uint(amax) >> 23);
          const int k = max(-126, min(126, 127 + 7 - ex));
          const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
          // (an infinite query has no such codes: its scores become NaN)
          if (lane == 0)
            ms->qs[seg % 3][h] =
                ex == 255 ? NAN : mul * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const int e = i * 32 + lane;
            if (e >= kPairs) continue;
            const float2 v = unpack_bf16x2(raw[j][i]);
            const float a = v.x * up, b = v.y * up;
            const uint32_t hi = lat::e4m3_pair(a, b);
            const float2 got = lat::e4m3_values(hi);
            const uint32_t lo = lat::e4m3_pair((a - got.x) * 16.f, (b - got.y) * 16.f);
            const int byte = 2 * e, c = byte >> 7, in = byte & 127;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              const int r = part * NH + h;
              const int at = c * C::kQChunkBytes + r * 128 + ((((in >> 4) ^ (r & 7)) << 4) | (in & 15));
              *reinterpret_cast<uint16_t*>(q_smem + at) = static_cast<uint16_t>(part == 0 ? hi : lo);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms->q_full);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      flag_error(err, PSW_DEVERR_PIPELINE);
    }
    // a copy in flight lands before the CTA ends
    if (!FP8 && seg > 0 && *abort_flag) mbar_wait(&ms->q_full, (seg - 1) & 1);
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loads
    // block id of page i of the segment; -1: zero rows
    auto block_id = [&](int i) -> int {
      if (i >= walk.seg_count) return -1;
      const int blk = pages.block_table[static_cast<int64_t>(walk.b) * pages.max_blocks +
                                        walk.span.first + walk.seg_first + i];
      if (blk >= 0 && blk < pages.num_blocks) return blk;
      flag_error(err, PSW_DEVERR_BLOCK_ID);
      return -1;
    };
    constexpr int kGroup = 32 / kPages;  // tiles whose block ids the lanes hold
    // TMA boxes of 16 rows x 128 bytes, issued by one lane of the converged warp
    // (issued by a lane each, a box costs 90 cycles: longer than it takes to
    // arrive). FP8 rows are 4.5 or 2.5 lines long and half of them straddle the
    // boxes' lines, which costs a gather of pages 6 % against whole pages.
    const bool one = lat::elect_one();
    uint32_t issued = 0;  // slots whose last load may be in flight, for the drain
    int tile = 0;
    bool stalled = false;  // testing hook: tile stall_tile of this CTA is never asked for
    while (ok && !stalled && walk.next()) {
      const int n_tiles = walk.tiles();
      int ids = block_id(lane), next_ids = block_id(32 + lane);
      for (int t = 0; ok && t < n_tiles; ++t, ++tile) {
        if (static_cast<int>(blockIdx.x) == stall_cta && tile == stall_tile) {
          stalled = true;  // leave quietly: the waits for it must run out
          break;
        }
        if (t > 0 && t % kGroup == 0) {
          ids = next_ids;
          next_ids = block_id((t / kGroup + 1) * 32 + lane);
        }
        int blk[kPages];
#pragma unroll
        for (int pg = 0; pg < kPages; ++pg)
          blk[pg] = __shfl_sync(0xffffffffu, ids, t % kGroup * kPages + pg);
#pragma unroll
        for (int u = 0; u <= C::kBlocks; ++u) {  // rope unit, then the blocks
          const int n = u == 0 ? 1 : C::kSlotsPerBlock;
          uint32_t parity;
          const int s = rg.take<C::kSlots>(n, parity);
#pragma unroll
          for (int c = 0; c < n; ++c) {
            ok = ok && mbar_wait(&ms->empty[s + c], (parity >> (s + c) & 1u) ^ 1u);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            issued |= 1u << (s + c);
            if (one) {
              uint64_t* full = &ms->full[s + c];
              mbar_arrive_expect_tx(full, kSlotBytes + (FP8 && u == 0 ? C::kScaleBytes : 0));
#pragma unroll
              for (int pg = 0; pg < kPages; ++pg) {
                lat::tma_box(smem_u32(ring + (s + c) * kSlotBytes + pg * 2048), &pool_map, full,
                             u == 0 ? LAT : (u - 1) * 128 + c * 64, blk[pg] * kBlockSize, 0);
                if (FP8 && u == 0)
                  lat::bulk_load(
                      smem_u32(scales + tile % C::kScaleTiles * C::kScaleBytes + pg * 64),
                      blk[pg] >= 0 ? static_cast<const void*>(pages.row_scale +
                                                              static_cast<int64_t>(blk[pg]) * kBlockSize)
                                   : g_zero_scales,
                      kBlockSize * 4, full);
              }
            }
          }
          if (!ok) break;
        }
        ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
      }
    }
    if ((!ok || stalled) && one) {
      if (!ok) {
        *abort_flag = 1;
        flag_error(err, PSW_DEVERR_PIPELINE);
      }
      // copies in flight land before the CTA ends: the last phase of each slot
      for (int s = 0; s < C::kSlots; ++s)
        if (issued >> s & 1u) mbar_wait(&ms->full[s], ((rg.phase >> s) & 1u) ^ 1u);
    }
  } else if (warp >= kScoreWarp) {
    // ------------------------------------------------------------ MMAs of S and of O
    // Two warps, so that neither product waits for the other's data. A warp
    // walks along converged and one lane issues; descriptors are a base, the
    // slot's place in it, and offsets known when compiling.
    const bool one = lat::elect_one();
    const uint64_t k_desc = tc::smem_desc(smem_u32(ring), 16, 1024, tc::kSwizzle128B);
    constexpr uint32_t kSlotStep = kSlotBytes >> 4;
    auto mma = [](uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
      if (FP8) lat::mma_ss_fp8(d, a, b, id, acc);
      else tc::mma_ss(d, a, b, id, acc);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && mbar_wait(bar, parity & 1u); };
    int seg = 0, tile = 0;
    for (; ok && walk.next(); ++seg) {
      const int n_tiles = walk.tiles();
      if (warp == kScoreWarp) wait(&ms->q_full, seg);
      ok = __all_sync(0xffffffffu, ok);
      for (int t = 0; ok && t < n_tiles; ++t, ++tile) {
        int slot[1 + C::kBlocks];
        uint32_t parity[1 + C::kBlocks];
#pragma unroll
        for (int u = 0; u <= C::kBlocks; ++u)
          slot[u] = rg.take<C::kSlots>(u == 0 ? 1 : C::kSlotsPerBlock, parity[u]);
        if (warp == kScoreWarp) {
          const uint32_t id_s = FP8 ? lat::idesc_e4m3_f32(kTile, C::kQRows, 0, 0)
                                    : tc::idesc_bf16_f32(kTile, C::kQRows, 0, 0);
          const uint64_t q_desc = tc::smem_desc(smem_u32(q_smem), 16, 1024, tc::kSwizzle128B);
          const uint32_t d = tmem + (tile & 1) * C::kQRows;
          // What this tile waits for: its slots; this buffer's S of two tiles ago has
          // been read; and the tile before that is over, so that no role is two phases
          // of a barrier behind. A wait takes ~100 cycles even for what is there: FP8
          // tiles mostly are, and all of it is first looked at by a lane each (37.5 ->
          // 36.7 us for three long sequences). bf16 tiles come just in time and would
          // be looked at in vain (67.6 -> 69.7 us for 32 sequences).
          uint32_t there = (tile < 2 ? 1u : 0u) << C::kTileSlots | (tile < 3 ? 2u : 0u) << C::kTileSlots;
          if constexpr (FP8) {
            uint64_t* bar = &ms->p_full[(tile + 1) % 3];
            uint32_t par = (tile - 2) / 3;
            if (lane == C::kTileSlots + 1) bar = &ms->pv_done[tile % 3], par = tile / 3 - 1;
#pragma unroll
            for (int u = 0; u <= C::kBlocks; ++u)
              if (lane == u) bar = &ms->full[slot[u]], par = parity[u] >> slot[u];
            static_assert(!FP8 || C::kTileSlots == C::kBlocks + 1, "a slot for each unit");
            there |= __ballot_sync(0xffffffffu, lane < C::kTileSlots + 2 && !(there >> lane & 1u) &&
                                                    mbar_test(bar, par & 1u));
            __syncwarp();
          }
          if (!(there >> C::kTileSlots & 1u)) wait(&ms->p_full[(tile + 1) % 3], (tile - 2) / 3);
          if (!(there >> (C::kTileSlots + 1) & 1u)) wait(&ms->pv_done[tile % 3], tile / 3 - 1);
#pragma unroll
          for (int u = 0; u <= C::kBlocks; ++u) {
#pragma unroll
            for (int c = 0; c < (u == 0 ? 1 : C::kSlotsPerBlock); ++c) {
              if (!(there >> (u == 0 ? 0 : 1 + (u - 1) * C::kSlotsPerBlock + c) & 1u))
                wait(&ms->full[slot[u] + c], parity[u] >> (slot[u] + c));
              tc::fence_after();
              const uint64_t kd = k_desc + (slot[u] + c) * kSlotStep;
              const uint64_t qd =
                  q_desc + static_cast<uint32_t>((u == 0 ? C::kQChunks - 1 : (u - 1) * C::kSlotsPerBlock + c) *
                                                 C::kQChunkBytes >> 4);
              if (ok && one) {
#pragma unroll
                for (int k = 0; k < (u == 0 ? C::kRopeSteps : 4); ++k)
                  mma(d, kd + k * 2, qd + k * 2, id_s, (u > 0 || k > 0) ? 1u : 0u);
              }
            }
          }
          if (ok && one) {
            tc::commit(&ms->s_full[tile & 1]);
            if (t == n_tiles - 1) tc::commit(&ms->q_free);
          }
        } else {
          const uint32_t id_o = FP8 ? lat::idesc_e4m3_f32(128, C::kPCols, 1, 1)
                                    : tc::idesc_bf16_f32(128, C::kPCols, 1, 1);
          const uint64_t v_desc = tc::smem_desc(smem_u32(ring), kSlotBytes, 1024, tc::kSwizzle128B);
          const uint64_t p_desc = tc::smem_desc(smem_u32(ring), 1024, 1024, tc::kSwizzle128B);
          // (P comes after S, and S after the tile has landed)
          wait(&ms->p_full[tile % 3], tile / 3);
          if (t == 0 && seg > 0) wait(&ms->o_free, seg - 1);
          tc::fence_after();
          const uint64_t pd = p_desc + slot[0] * kSlotStep;
          if (ok && one) {
#pragma unroll
            for (int m = 0; m < C::kBlocks; ++m) {
              const uint64_t vd = v_desc + slot[1 + m] * kSlotStep;
#pragma unroll
              for (int k = 0; k < C::kPSteps; ++k) {
                constexpr uint32_t kStep = C::kPStepBytes >> 4;
                mma(tmem + C::kTmemO + m * C::kPCols, vd + k * kStep, pd + k * kStep, id_o,
                    (t > 0 || k > 0) ? 1u : 0u);
              }
#pragma unroll
              for (int c = 0; c < C::kSlotsPerBlock; ++c) tc::commit(&ms->empty[slot[1 + m] + c]);
            }
            tc::commit(&ms->empty[slot[0]]);
            tc::commit(&ms->pv_done[tile % 3]);
            if (t == n_tiles - 1) tc::commit(&ms->o_full);
          }
        }
        ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
      }
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
    const int row_warp = warp & 3, head0 = (warp >> 2) * 16;  // which rows, which heads
    const uint32_t lanes = static_cast<uint32_t>(row_warp * 32) << 16;
    const float cap2 = softcap * lat::kLog2e;
    // this thread's keys of a tile, rows 16 row_warp + lane / 4 and 8 further; its
    // heads head0 + 8 g + 2 (lane mod 4) + {0, 1}, number 2 g + {0, 1} here
    const int r0 = row_warp * 16 + (lane >> 2), quad = lane & 3;
    auto head_of = [&](int i) { return head0 + 8 * (i >> 1) + 2 * quad + (i & 1); };
    // Before anything else a CTA goes through the tile's code once without
    // effect (segment -1): fetching that code costs 1200 (bf16) to 5000 (FP8)
    // cycles, several times that behind the first loads, now none of them of the
    // first tile's.
    int seg = -1, tile = 0;
    bool more = true;
    Walk w = {};
    for (; ok && more; ++seg) {
      if (seg >= 0) {
        w = walk;
        more = walk.next();
      }
      const int h0 = w.chunk * NH, nh = min(NH, heads - h0), n_tiles = w.tiles();
      constexpr int HN = C::kHeads;
      // FP8: ref is the log2 of the unit
      float m[HN], l[HN], ref[HN];
      // FP8: the unit of some head is coarse for a row if log2 of its scale is below `fine`
      float fine = -INFINITY;
      const float spare = C::kSpare - __log2f(static_cast<float>(w.seg_count * kBlockSize));
#pragma unroll
      for (int i = 0; i < HN; ++i) m[i] = 0.f, l[i] = 0.f, ref[i] = 0.f;
      for (int t = seg < 0 ? -1 : 0; t < n_tiles; ++t) {
        const bool live = t >= 0;
        const bool in_seg = live && t * kPages + row_warp < w.seg_count;  // a page per warp
        const int key = (w.span.first + w.seg_first + t * kPages + row_warp) * kBlockSize + (lane >> 2);
        int slot[1 + C::kBlocks] = {};
        uint32_t parity[1 + C::kBlocks] = {};
        if (live) {
#pragma unroll
          for (int u = 0; u <= C::kBlocks; ++u)
            slot[u] = rg.take<C::kSlots>(u == 0 ? 1 : C::kSlotsPerBlock, parity[u]);
          ok = mbar_wait(&ms->s_full[tile & 1], (tile >> 1) & 1);
          tc::fence_after();
        }
        bool seen[2];
        float vs[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          seen[j] = in_seg && key + 8 * j >= w.span.lo && key + 8 * j < w.span.len;
          // the row's scale (it landed with the rope unit, whose phase every
          // reader looks at itself); a hidden slot's may be anything
          if (FP8 && j == 0 && live) ok = ok && mbar_wait(&ms->full[slot[0]], parity[0] >> slot[0] & 1u);
          vs[j] = FP8 && seen[j]
                      ? reinterpret_cast<const float*>(scales + (tile % C::kScaleTiles) * C::kScaleBytes)[r0 + 8 * j]
                      : 0.f;
        }
        float z[2][HN];
        {
          uint32_t v[C::kQParts][8];
#pragma unroll
          for (int p = 0; p < C::kQParts; ++p)
            lat::ld16x256_x2(tmem + lanes + (tile & 1) * C::kQRows + p * NH + head0, v[p]);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < HN; ++i) {
            const int r = 4 * (i >> 1) + (i & 1);
            const float qs = FP8 ? ms->qs[(seg + 3) % 3][head_of(i)] : mul;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float x = __uint_as_float(v[0][r + 2 * j]);
              z[j][i] = FP8 ? fmaf(__uint_as_float(v[C::kQParts - 1][r + 2 * j]), 0.0625f, x) * (qs * vs[j])
                            : x * qs;
            }
          }
        }
        if (softcap > 0.f) {
#pragma unroll
          for (int i = 0; i < HN; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              z[j][i] = cap2 * (FAR_CAP ? lat::tanh_of(z[j][i]) : lat::tanh_large(z[j][i]));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int i = 0; i < HN; ++i) z[j][i] = seen[j] ? z[j][i] : -INFINITY;
          // rows of a loaded page that hold no visible key must not enter the
          // second product (P is 0 there, but 0 times NaN is not)
          if (in_seg && !seen[j] && head0 == 0) {
#pragma unroll
            for (int u = 1; u <= C::kBlocks; ++u)
              for (int c = 0; c < C::kSlotsPerBlock; ++c) {
                ok = ok && mbar_wait(&ms->full[slot[u] + c], parity[u] >> (slot[u] + c) & 1u);
                for (int i = 0; i < 2; ++i)
                  *reinterpret_cast<uint4*>(ring + (slot[u] + c) * kSlotBytes + (r0 + 8 * j) * 128 +
                                            quad * 32 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
          }
        }
        float over = -INFINITY, hi = -INFINITY, lo = INFINITY;
#pragma unroll
        for (int i = 0; i < HN; ++i) {
          const float x = fmaxf(z[0][i], z[1][i]);
          over = fmaxf(over, x - m[i]);
          if (FP8) hi = fmaxf(hi, x - ref[i]), lo = fminf(lo, x - ref[i]);
        }
        bool move = !ok || t <= 0 || over > C::kLag;
        // FP8: log2 of the rows' scales, and whether a unit may have to move. One that is too
        // coarse is so for a key of some warp, in which then each of the eight lanes of that
        // head finds its two keys small; and a thread's two keys are not told apart here. Where
        // that says yes, all warps look head by head.
        float lv[2];
        uint32_t anew = 0;  // of this warp's heads: small and coarse
        if constexpr (FP8) {
          lv[0] = __log2f(fabsf(vs[0]));
          lv[1] = __log2f(fabsf(vs[1]));
          move |= hi + fmaxf(lv[0], lv[1]) > C::kMost;
          if (__any_sync(0xffffffffu, (lv[0] > -INFINITY && lv[0] < fine) ||
                                          (lv[1] > -INFINITY && lv[1] < fine))) {
            uint32_t b = __ballot_sync(0xffffffffu, lo + fminf(lv[0], lv[1]) < C::kLeast);
            b &= b >> 16;
            b &= b >> 8;
            b &= b >> 4;
            move |= (b & 15u) != 0;
          }
        }
        bool settle = lat::bar_any(1, kSoftThreads, move);
        if constexpr (FP8) {
          if (settle) {
            move = !ok || t <= 0 || over > C::kLag;
            uint32_t says = 0;
#pragma unroll
            for (int i = 0; i < HN; ++i) {
              const float at = fmaxf(z[0][i] + lv[0], z[1][i] + lv[1]) - ref[i];
              const float least = ref[i] - m[i] - spare;
              move |= at > C::kMost;
              says |= at >= C::kLeast ? 1u << i : 0u;
              says |= (lv[0] > -INFINITY && lv[0] < least) || (lv[1] > -INFINITY && lv[1] < least)
                          ? 0x10000u << i
                          : 0u;
            }
            says = __reduce_or_sync(0xffffffffu, says << (4 * quad));
            const bool up = __any_sync(0xffffffffu, move);
            if (lane == 0) {
              ms->says[warp] = says;
              ms->up[warp] = up;
            }
            named_bar_sync(1, kSoftThreads);
            settle = false;
#pragma unroll
            for (int k = 0; k < C::kGroups; ++k) {
              const uint4 a4 = *reinterpret_cast<const uint4*>(&ms->says[4 * k]);
              const uint4 u4 = *reinterpret_cast<const uint4*>(&ms->up[4 * k]);
              const uint32_t of = (a4.x | a4.y) | (a4.z | a4.w);
              settle |= ((u4.x | u4.y) | (u4.z | u4.w) | (of >> 16 & ~of)) != 0;
              if (k == warp >> 2) anew = of >> 16 & ~of;
            }
          }
        }
        if (settle) {
          // the tile's maxima; the ones in use move to them where they lag
#pragma unroll
          for (int i = 0; i < HN; ++i) {
            float x = fmaxf(z[0][i], z[1][i]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            if (lane < 4) ms->red[row_warp][head_of(i)] = x;
          }
          if constexpr (FP8) {  // and the largest weights
#pragma unroll
            for (int i = 0; i < HN; ++i) {
              float x = fmaxf(z[0][i] + lv[0], z[1][i] + lv[1]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
              if (lane < 4) ms->heavy[row_warp][head_of(i)] = x;
            }
          }
          named_bar_sync(1, kSoftThreads);
          float a[HN], top[HN];
          bool moved = false;
#pragma unroll
          for (int i = 0; i < HN; ++i) {
            const int h = head_of(i);
            const float x = fmaxf(fmaxf(ms->red[0][h], ms->red[1][h]), fmaxf(ms->red[2][h], ms->red[3][h]));
            a[i] = 1.f;
            if (t <= 0) {
              l[i] = 0.f;
              m[i] = x == -INFINITY ? 0.f : x;
            } else if (x > m[i] + (FP8 ? 0.f : C::kLag)) {  // (FP8: O does not depend on it)
              a[i] = ex2_approx(m[i] - x);
              l[i] *= a[i];
              m[i] = x;
            }
          }
          if constexpr (FP8) {
            fine = -INFINITY;
#pragma unroll
            for (int i = 0; i < HN; ++i) {
              const int h = head_of(i);
              const float x = fmaxf(fmaxf(ms->heavy[0][h], ms->heavy[1][h]), fmaxf(ms->heavy[2][h], ms->heavy[3][h]));
              const float old = ref[i];
              top[i] = t <= 0 ? x : fmaxf(ms->top[h], x);
              if (t <= 0) {
                ref[i] = x > -INFINITY ? x - C::kAim : m[i];
              } else if (x > -INFINITY &&
                         (x - old > C::kMost || (anew >> (4 * quad + i) & 1u) != 0)) {
                // (by a power of two, so that O keeps its bits)
                ref[i] = fmaxf(old + rintf(x - C::kAim - old), top[i] - (C::kAim + C::kReach));
              }
              fine = fmaxf(fine, ref[i] - m[i] - spare);
              a[i] = ex2_approx(fminf(old - ref[i], 100.f));  // (beyond: O is still zero)
            }
          }
#pragma unroll
          for (int i = 0; i < HN; ++i) {
            moved |= a[i] != 1.f;
            if (row_warp == 0 && lane < 4) ms->alpha[head_of(i)] = a[i];
          }
          moved = lat::bar_any(1, kSoftThreads, !ok || (t > 0 && moved));
          if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < HN; ++i)
              if (row_warp == 0 && lane < 4) ms->top[head_of(i)] = top[i];
          }
          if (moved) {
            // O is rescaled: the products up to the tile before have ended
            if (t > 0) {
              ok = __all_sync(0xffffffffu, ok && mbar_wait(&ms->pv_done[(tile - 1) % 3], (tile - 1) / 3 & 1));
              if (ok) {
                tc::fence_after();
                const float f = FP8 && lane < NH ? ms->alpha[lane] : 1.f;
                const uint32_t heads_moved = __ballot_sync(0xffffffffu, f != 1.f);
                if (FP8 && __popc(heads_moved) <= kFewHeads) {  // their columns alone
                  for (uint32_t left = heads_moved; left != 0; left &= left - 1) {
                    const int h = __ffs(static_cast<int>(left)) - 1;
                    const float by = __shfl_sync(0xffffffffu, f, h);
                    constexpr int kMine = C::kBlocks / C::kGroups * C::kPParts;
                    uint32_t v[kMine];
                    auto at = [&](int k) {
                      return tmem + lanes + C::kTmemO + h +
                             ((warp >> 2) + k / C::kPParts * C::kGroups) * C::kPCols +
                             k % C::kPParts * NH;
                    };
#pragma unroll
                    for (int k = 0; k < kMine; ++k) lat::ld1(at(k), v[k]);
                    tc::wait_ld();
#pragma unroll
                    for (int k = 0; k < kMine; ++k)
                      lat::st1(at(k), __float_as_uint(__uint_as_float(v[k]) * by));
                  }
                } else {
#pragma unroll 1
                  for (int blk = warp >> 2; blk < C::kBlocks; blk += C::kGroups) {
#pragma unroll
                    for (int c = 0; c < C::kPCols / 16; ++c) {
                      uint32_t v[16];
                      const uint32_t at = tmem + lanes + C::kTmemO + blk * C::kPCols + c * 16;
                      tc::ld16(at, v);
                      tc::wait_ld();
#pragma unroll
                      for (int i = 0; i < 16; ++i)
                        v[i] = __float_as_uint(__uint_as_float(v[i]) * ms->alpha[(c * 16 + i) % NH]);
                      tc::st16(at, v);
                    }
                  }
                }
                tc::wait_st();
              }
            }
            if (lat::bar_any(1, kSoftThreads, !ok)) {  // (and alpha may be written again)
              ok = false;
              break;
            }
          }
        }
        // P into the rope slot: a key's row holds the parts of all heads,
        // 16-byte vectors swizzled by the row
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = r0 + 8 * j, sw = r & 7;
          uint8_t* prow = ring + slot[0] * kSlotBytes + r * 128;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float a = ex2_approx(z[j][2 * g] - m[2 * g]);
            float b = ex2_approx(z[j][2 * g + 1] - m[2 * g + 1]);
            l[2 * g] += a;
            l[2 * g + 1] += b;
            if (!FP8) {
              const uint32_t hi = pack_bf16x2(a, b);
              const float2 got = unpack_bf16x2(hi);
              if (!live) continue;
              const int vec = (head0 >> 3) + g;
              *reinterpret_cast<uint32_t*>(prow + ((vec ^ sw) << 4) + quad * 4) = hi;
              *reinterpret_cast<uint32_t*>(prow + (((vec + NH / 8) ^ sw) << 4) + quad * 4) =
                  pack_bf16x2(a - got.x, b - got.y);
            } else {
              a = copysignf(ex2_approx(z[j][2 * g] + lv[j] - ref[2 * g]), vs[j]);
              b = copysignf(ex2_approx(z[j][2 * g + 1] + lv[j] - ref[2 * g + 1]), vs[j]);
#pragma unroll
              for (int p = 0; p < 3; ++p) {
                const uint32_t c = lat::e4m3_pair(a, b);
                const int at = p * NH + head0 + g * 8 + quad * 2;
                if (live)
                  *reinterpret_cast<uint16_t*>(prow + (((at >> 4) ^ sw) << 4) + (at & 15)) =
                      static_cast<uint16_t>(c);
                const float2 got = lat::e4m3_values(c);
                a = (a - got.x) * 16.f;
                b = (b - got.y) * 16.f;
              }
            }
          }
        }
        fence_proxy_async_smem();
        tc::fence_before();
        __syncwarp();
        if (live) {
          if (lane == 0) mbar_arrive(&ms->p_full[tile % 3]);
          ++tile;
        }
      }
      if (!ok) break;
      if (seg < 0) {
        wait_for_inputs();
        named_bar_sync(4, kSoftThreads + 32);
        begin();
        more = walk.next();
        continue;
      }
      // ---- the segment's end
#pragma unroll
      for (int i = 0; i < C::kHeads; ++i) {
        float x = l[i];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        const int h = head_of(i);
        if (lane < 4) ms->red[row_warp][h] = x;
        if (row_warp == 0 && lane < 4) {
          ms->alpha[h] = m[i];
          if (FP8) ms->top[h] = ex2_approx(0.5f * (ref[i] - m[i]));
        }
      }
      ok = mbar_wait(&ms->o_full, seg & 1);
      if (lat::bar_any(1, kSoftThreads, !ok)) {
        ok = false;
        break;
      }
      tc::fence_after();
      const bool whole = w.whole();
      const int slot_id = 2 * blockIdx.x + (w.seg_first == 0 ? 1 : 0);
      if (tid < nh) {  // thread h: the statistics of head h
        const float mh = ms->alpha[tid];
        const float s = ms->red[0][tid] + ms->red[1][tid] + ms->red[2][tid] + ms->red[3][tid];
        ms->lsum[tid] = (whole ? (s == 0.f ? 0.f : 1.f / s) : 1.f) * (FP8 ? ms->top[tid] : 1.f);
        if (whole) {
          if (lse != nullptr)
            lse[static_cast<int64_t>(w.b) * heads + h0 + tid] = (mh + __log2f(s)) * lat::kLn2;
        } else {
          part_ml[slot_id * kMaxHeads + tid] = make_float2(mh, s);
        }
      }
      if (tid == 0 && w.seg_first == 0) {
        // first page of the unit: note which pieces share it (the segment ends
        // where w.left is left of this piece)
        const int end = ms->p1 - w.left - w.seg_count + w.span.count;  // list end of the unit
        const int last = ms->cut.piece(end - 1);
        parts[w.b * chunks + w.chunk] = whole ? Part{-1, -1} : Part{static_cast<int32_t>(blockIdx.x), last};
      }
      named_bar_sync(1, kSoftThreads);
#pragma unroll 1
      for (int blk = warp >> 2; blk < C::kBlocks; blk += C::kGroups) {
        const int d = blk * 128 + row_warp * 32 + lane;
        float o[NH];
#pragma unroll
        for (int p = 0; p < C::kPParts; ++p) {
          uint32_t v[NH];
#pragma unroll
          for (int c = 0; c < NH / 16; ++c)
            tc::ld16(tmem + lanes + C::kTmemO + blk * C::kPCols + p * NH + c * 16,
                     *reinterpret_cast<uint32_t(*)[16]>(&v[c * 16]));
          tc::wait_ld();
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const float x = __uint_as_float(v[h]);
            o[h] = p == 0 ? x : fmaf(x, FP8 ? (p == 1 ? 0.0625f : 0.00390625f) : 1.f, o[h]);
          }
        }
        if (whole) {
          __nv_bfloat16* dst = out + (static_cast<int64_t>(w.b) * heads + h0) * LAT + d;
#pragma unroll
          for (int h = 0; h < NH; ++h)
            if (h < nh) dst[h * LAT] = __float2bfloat16_rn((FP8 ? o[h] * ms->top[h] : o[h]) * ms->lsum[h]);
        } else {
          float* dst = part_o + static_cast<int64_t>(slot_id) * kMaxHeads * LAT + d;
#pragma unroll
          for (int h = 0; h < NH; ++h)
            if (h < nh) dst[h * LAT] = FP8 ? o[h] * ms->top[h] * ms->lsum[h] : o[h];
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->o_free);
      named_bar_sync(1, kSoftThreads);  // red and lsum may be written again
    }
    if (!ok) {
      if (tid == 0) {
        *abort_flag = 1;
        flag_error(err, PSW_DEVERR_PIPELINE);
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == kScoreWarp) tc::dealloc(tmem, 512);
}

// Joins what the pieces of a unit left: out = sum_i 2^(m_i - M) O_i / sum_i
// 2^(m_i - M) l_i. One CTA per (sequence, head); a group of L / 4 threads, four
// dims each, takes every groups-th piece, and the groups' sums meet in shared
// memory. The kernel is a chain of three loads (lengths, which pieces, then
// statistics and the first eight pieces together). A unit that one piece covered
// is left alone, an empty sequence gets its zeros. Where a wait of the first kernel
// ran out, what it should have noted was not: the workspace may hold anything there, so
// pieces that the first kernel does not have are flagged and their unit is left alone.
constexpr int kMergeThreads = 512;
template <int LAT>
__global__ void __launch_bounds__(kMergeThreads)
latent_merge_kernel(const int32_t* seq_lens, int heads, int max_pieces, const Part* parts,
                    const float2* part_ml, const float* part_o, __nv_bfloat16* __restrict__ out,
                    float* __restrict__ lse, int32_t* err) {
  constexpr int kRow = LAT / 4;  // threads of a group
  __shared__ float s_w[kMergeThreads / 32][kMaxCtas];
  __shared__ float4 s_o[kMergeThreads];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int group = tid / kRow, groups = blockDim.x / kRow, col = tid - group * kRow;
  const int nh = chunk_heads(heads), chunk = h / nh, hc = h - chunk * nh;
  const int64_t row = static_cast<int64_t>(b) * heads + h;
  uint2* dst = reinterpret_cast<uint2*>(out + row * LAT) + col;
  wait_for_inputs();
  const int len = seq_lens[b];
  const Part pt = len > 0 ? parts[b * chunks_of(heads) + chunk] : Part{-1, -1};
  if (len <= 0) {
    if (group == 0) *dst = make_uint2(0u, 0u);
    if (lse != nullptr && tid == 0) lse[row] = -INFINITY;
    return;
  }
  if (pt.x < 0) return;
  if (pt.y < pt.x || pt.y >= max_pieces) {
    if (tid == 0) flag_error(err, PSW_DEVERR_PIPELINE);
    return;
  }
  const int n = pt.y - pt.x + 1;  // at most max_pieces, which is at most kMaxCtas
  auto slot = [&](int i) { return i == 0 ? 2 * pt.x + 1 : 2 * (pt.x + i); };
  auto piece = [&](int i) -> float4 {
    return i < n ? __ldcg(reinterpret_cast<const float4*>(
                              part_o + (static_cast<int64_t>(slot(i)) * kMaxHeads + hc) * LAT) +
                          col)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = piece(group + k * groups);
  // every warp forms the pieces' weights by itself
  float2 ml[kMaxCtas / 32];
  float mx = -INFINITY, l = 0.f;
#pragma unroll
  for (int k = 0; k < kMaxCtas / 32; ++k) {
    const int i = lane + k * 32;
    ml[k] = i < n ? __ldcg(part_ml + slot(i) * kMaxHeads + hc) : make_float2(-INFINITY, 0.f);
    mx = fmaxf(mx, ml[k].x);
  }
  mx = lat::warp_max(mx);
  float* w = s_w[tid >> 5];
#pragma unroll
  for (int k = 0; k < kMaxCtas / 32; ++k) {
    const int i = lane + k * 32;
    const float x = i < n ? ex2_approx(ml[k].x - mx) : 0.f;
    w[i] = x;
    l = fmaf(x, ml[k].y, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  __syncwarp();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = group; i0 < n; i0 += 8 * groups) {
    if (i0 != group) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = piece(i0 + k * groups);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = i0 + k * groups < n ? w[i0 + k * groups] : 0.f;
      acc.x = fmaf(x, v[k].x, acc.x);
      acc.y = fmaf(x, v[k].y, acc.y);
      acc.z = fmaf(x, v[k].z, acc.z);
      acc.w = fmaf(x, v[k].w, acc.w);
    }
  }
  if (groups > 1) {
    s_o[tid] = acc;
    __syncthreads();
    if (group != 0) return;
    for (int g = 1; g < groups; ++g) {
      const float4 x = s_o[g * kRow + col];
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *dst = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lse != nullptr && tid == 0) lse[row] = (mx + __log2f(l)) * lat::kLn2;
}

struct Layout {
  size_t ml, o, total;
};
Layout layout(const LatentArgs& L, int n_seqs) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Layout y;
  y.ml = up(sizeof(Part) * static_cast<size_t>(n_seqs) * chunks_of(L.n_heads));
  y.o = y.ml + up(sizeof(float2) * 2 * kMaxCtas * kMaxHeads);
  y.total = y.o + sizeof(float) * 2 * kMaxCtas * kMaxHeads * static_cast<size_t>(L.latent);
  return y;
}

template <int LAT, int NH, bool FP8>
int launch(const LatentArgs& L, const void* q, const LatentPages& pages, const int32_t* seq_lens,
           int n_seqs, void* out, float* lse, void* ws, int num_sms, int32_t* err,
           cudaStream_t stream) {
  using C = Cfg<LAT, NH, FP8>;
  CUtensorMap q_map, pool_map;
  const int row = L.row();
  int rc = make_map_3d(&q_map, false, q, {row, L.n_heads, n_seqs},
                       {int64_t{2} * row, int64_t{2} * row * L.n_heads}, {64, NH, 1});
  if (rc != PSW_OK) return rc;
  const int64_t row_bytes = FP8 ? row : 2 * row;
  rc = make_map_3d(&pool_map, FP8, pages.pool, {row, pages.num_blocks * kBlockSize, 1},
                   {row_bytes, row_bytes},
                   {C::kElems, kBlockSize, 1});
  if (rc != PSW_OK) return rc;
  // (as a run-time choice the form for large caps cost the others 1 to 10 %)
  auto* kernel = L.softcap > lat::kNearCap ? latent_decode_kernel<LAT, NH, FP8, true>
                                           : latent_decode_kernel<LAT, NH, FP8, false>;
  rc = set_smem_limit(reinterpret_cast<const void*>(kernel), C::kSmemBytes);
  if (rc != PSW_OK) return rc;
  const Layout y = layout(L, n_seqs);
  auto* base = static_cast<uint8_t*>(ws);
  auto* parts = reinterpret_cast<Part*>(base);
  auto* ml = reinterpret_cast<float2*>(base + y.ml);
  auto* o = reinterpret_cast<float*>(base + y.o);
  auto* ob = static_cast<__nv_bfloat16*>(out);
  const int grid = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const StallHook stall = stall_hook(kStallDecode);
  if (cudaLaunchKernelEx(&cfg, kernel, q_map, pool_map, pages,
                         static_cast<const __nv_bfloat16*>(q), seq_lens, n_seqs, L.n_heads,
                         L.window, L.scale, L.softcap, ob, lse, parts, ml, o, err, stall.cta,
                         stall.tile) != cudaSuccess)
    return PSW_ELAUNCH;
  cfg.gridDim = dim3(n_seqs, L.n_heads);
  cfg.dynamicSmemBytes = 0;
  // pieces a unit has on average, eight loads in flight per group of threads
  const int64_t units = static_cast<int64_t>(n_seqs) * chunks_of(L.n_heads);
  const int row_threads = L.latent / 4;
  const int want = static_cast<int>(1 + (grid / units) / 8);
  const int fit = kMergeThreads / row_threads;
  cfg.blockDim = dim3(row_threads * (want < fit ? want : fit));
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, latent_merge_kernel<LAT>, seq_lens, L.n_heads, grid,
      static_cast<const Part*>(parts), static_cast<const float2*>(ml),
      static_cast<const float*>(o), ob, lse, err);
  return e == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

}  // namespace ldec

size_t latent_decode_workspace(const LatentArgs& L, int n_seqs) {
  return ldec::layout(L, n_seqs).total;
}

int launch_latent_decode(const LatentArgs& L, const void* q, const LatentPages& pages,
                         const int32_t* seq_lens, int n_seqs, void* out, float* lse, void* ws,
                         int num_sms, int32_t* err, cudaStream_t stream) {
#define PSW_PICK(LAT_, NH_)                                                                       \
  (pages.row_scale != nullptr                                                                     \
       ? ldec::launch<LAT_, NH_, true>(L, q, pages, seq_lens, n_seqs, out, lse, ws, num_sms, err, \
                                       stream)                                                    \
       : ldec::launch<LAT_, NH_, false>(L, q, pages, seq_lens, n_seqs, out, lse, ws, num_sms,     \
                                        err, stream))
  const bool few = ldec::chunk_heads(L.n_heads) == 16;
  if (L.latent == 512) return few ? PSW_PICK(512, 16) : PSW_PICK(512, 32);
  return few ? PSW_PICK(256, 16) : PSW_PICK(256, 32);
#undef PSW_PICK
}

}  // namespace psw
