// latent_expand.cu -- cached latent rows read back from their pages and
// expanded to every head's key and value components:
//   kv[t][h][e] = sum_l c_l w[h][e][l],  k_rope[t] = r.
// A matrix product of gathered rows, 512 or 1024 operations per output byte:
// bound by the tensor cores, beside writing 512 bytes per row and head.
//
// Schedule: the list of units (256 rows, a head, keys or values: 128 outputs of
// each row) is cut evenly over pairs of CTAs, whose tensor cores share products of
// 256 rows x 128 outputs: each CTA holds half of the rows, in tensor memory (A of
// the products: 128 lanes x L / 2 columns), and loads half of the outputs' rows of w
// (warp 5, TMA, boxes of 64 x 128 columns), so that a byte of w in shared memory
// serves 256 rows. Warp 4 of the first CTA issues for both, into two accumulators;
// the second's tells it what of w has landed there. Warps 0-3 round, turn the rows
// around through shared memory and write 64-byte pieces. Warps 6-9 gather rows:
// rows of a tile are any rows of any pages, so they are copied 16 bytes at a time
// (asynchronously; FP8 codes are exact in bf16 and are converted on the way, the
// row's scale multiplies the fp32 result) into shared memory, four chunks of 64
// columns ahead, and moved into tensor memory chunk by chunk as the last unit of the
// tile before is done with them.
//
// Measured: 40k rows of 16 heads, latent 512, 170 GFLOP: 106 us in a graph of twelve
// calls, 109 by itself (1.55 PFLOP/s, 79 % of the measured bf16 rate; the tensor cores
// are active 78 % of the time), 120 in a long run of calls on changing inputs. A
// unit takes ~2330 cycles where its 32 products of 68 cycles take 2176; 13000 cycles
// pass before the first (20 MB are gathered at once), 3000 to 6000 from one
// tile to the next. What was slower: rows in shared memory (144 us: that memory's
// 128 bytes a cycle are then the bound), products of one CTA with w sent to both of a
// pair (129), the whole of the next tile's rows ahead with a smaller ring of w
// (115: w at 30 bytes a cycle is all that L2 gives an SM, and rows come slower still).
#include "latent.cuh"

namespace psw {
namespace lexp {

constexpr int kTile = 128;
constexpr int kUnit = kTile * 128;              // bytes of a chunk of rows
constexpr int kBoxChunks = 2;                   // chunks of a box of w
constexpr int kBox = kBoxChunks * kUnit / 2;    // bytes of a CTA's half of one
constexpr int kMmaWarp = 4, kWeightWarp = 5, kRowWarp = 6;
constexpr int kRowThreads = 128;                // warps 6-9
constexpr int kThreads = 320;
constexpr int kAcc = 2;                         // accumulators of 128 columns
constexpr int kStage = 4 * 32 * 64;             // epilogue: 32 rows x 64 B per warp
constexpr int kMisc = 4096;
constexpr int kAhead = 4;                       // chunks of rows in shared memory
constexpr int kCluster = 2;
constexpr int kMaxRing = 9;
constexpr int kSmemLimit = 232448;

template <int LAT>
struct Cfg {
  static constexpr int kChunks = LAT / 64;
  static constexpr int kRing = (kSmemLimit - 1024 - kMisc - kStage - kAhead * kUnit) / kBox;
  static constexpr int kSmemBytes = 1024 + kAhead * kUnit + kRing * kBox + kStage + kMisc;
  static_assert(kChunks % kAhead == 0, "rows come in groups of chunks");
  static_assert(kRing >= 4 && kRing <= kMaxRing, "boxes of w in flight");
  static constexpr int kTmemD = LAT / 2;          // after the rows
  static_assert(kTmemD + kAcc * kTile <= 512, "tensor memory columns");
};

struct Misc {
  uint64_t a_full[8], a_empty[8], w_full[kMaxRing], w_empty[kMaxRing], d_full[kAcc], d_empty[kAcc];
  uint64_t rows_done[2], rows_set[2], drained;
  uint32_t tmem;
  int32_t abort;
  int32_t slot[2][kTile];   // pool slot of each row of a tile, -1: a zero row; tiles in turn
  float scale[2][kTile];
};
static_assert(sizeof(Misc) <= kMisc, "misc block");

template <int LAT, bool FP8>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
latent_expand_kernel(const __grid_constant__ CUtensorMap w_map, const LatentPages pages,
                     const int32_t* __restrict__ cu_k, const int32_t* __restrict__ k_first,
                     int n_seqs, int n_k, int heads, __nv_bfloat16* __restrict__ kv,
                     __nv_bfloat16* __restrict__ k_rope, int32_t* err) {
  using C = Cfg<LAT>;
  constexpr int kRow = LAT + kLatentRope;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* a_smem = smem;  // rows on their way
  uint8_t* w_ring = smem + kAhead * kUnit;
  uint8_t* stage = w_ring + C::kRing * kBox;
  Misc* ms = reinterpret_cast<Misc*>(stage + kStage);

  if (warp == kMmaWarp) {
    lat::alloc_pair(&ms->tmem, 512);
  }
  const uint32_t rank = lat::cluster_rank();
  if (tid == 0) {
    // (the first CTA issues the products of both: what they wait for arrives there)
    for (int i = 0; i < 8; ++i) {
      mbar_init(&ms->a_full[i], 4 * kCluster);
      mbar_init(&ms->a_empty[i], 1);
    }
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&ms->w_full[i], rank == 0 ? kCluster : 1);
      mbar_init(&ms->w_empty[i], 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(&ms->d_full[i], 1);
      mbar_init(&ms->d_empty[i], 4 * kCluster);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms->rows_set[i], 4);
      mbar_init(&ms->rows_done[i], 4);
    }
    mbar_init(&ms->drained, 1);
    ms->abort = 0;
    fence_mbar_init();
  }
  __syncwarp();
  tc::fence_before();
  lat::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = ms->tmem;
  volatile int32_t* abort_flag = &ms->abort;
  const int named = __ldg(cu_k + n_seqs), total = max(0, min(n_k, named));
  if (named > n_k && blockIdx.x == 0 && tid == 0) flag_error(err, PSW_DEVERR_LENGTH);
  const int per_tile = heads * 2;
  const int pair = blockIdx.x / kCluster, pairs = gridDim.x / kCluster;
  const int64_t units =
      (static_cast<int64_t>(total) + kCluster * kTile - 1) / (kCluster * kTile) * per_tile;
  const int64_t u0 = units * pair / pairs, u1 = units * (pair + 1) / pairs;
  // tile n of this CTA is number kCluster (first_tile + n) + rank
  const int first_tile = static_cast<int>(u0 / per_tile);
  const int first_sub = static_cast<int>(u0 - static_cast<int64_t>(first_tile) * per_tile);
  const int count = static_cast<int>(u1 - u0);
  bool ok = true;

  if (count == 0) {
    // nothing to do
  } else if (warp >= kRowWarp) {
    // ------------------------------------------------------------ rows
    const int t = tid - kRowWarp * 32, rw = warp - kRowWarp;
    const int n_tiles = (first_sub + count + per_tile - 1) / per_tile;
    const int r = (warp & 3) * 32 + lane;  // this warp's lanes of tensor memory are these rows
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint4 raw[kAhead][4];  // FP8: the codes of a group of chunks

    // where each row of tile n lives
    auto locate = [&](int n) {
      const int64_t row0 = (static_cast<int64_t>(first_tile + n) * kCluster + rank) * kTile;
      const int buf = n & 1;
      // (the results of two tiles ago are written: its scales are done with)
      if (n >= 2) ok = ok && mbar_wait(&ms->rows_done[buf], ((n >> 1) - 1) & 1);
      int64_t slot = -1;
      if (row0 + t < total) {
        const int row = static_cast<int>(row0) + t;
        int lo = 0, hi = n_seqs;  // the largest b with cu_k[b] <= row
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(cu_k + mid) <= row) lo = mid;
          else hi = mid;
        }
        const int start = __ldg(cu_k + lo), end = __ldg(cu_k + lo + 1);
        const int first = k_first != nullptr ? __ldg(k_first + lo) : 0;
        const int64_t pos = static_cast<int64_t>(first) + (row - start);
        int32_t bits = 0;
        if (row < start || row >= end || first < 0) {
          bits = PSW_DEVERR_LENGTH;
        } else if (pos / kBlockSize >= pages.max_blocks) {
          bits = PSW_DEVERR_CAPACITY;
        } else {
          const int32_t blk = __ldg(pages.block_table + static_cast<int64_t>(lo) * pages.max_blocks +
                                    pos / kBlockSize);
          if (blk < 0 || blk >= pages.num_blocks) bits = PSW_DEVERR_BLOCK_ID;
          else slot = static_cast<int64_t>(blk) * kBlockSize + pos % kBlockSize;
        }
        if (bits != 0) flag_error(err, bits);
      }
      ms->slot[buf][t] = static_cast<int32_t>(slot);
      if (FP8) ms->scale[buf][t] = slot >= 0 ? __ldg(pages.row_scale + slot) : 0.f;
      named_bar_sync(1, kRowThreads);
      if (lane == 0) mbar_arrive(&ms->rows_set[buf]);
    };
    // chunk c of the rows in slots: on its way (bf16: to shared memory, a copy group;
    // FP8: to registers)
    auto start = [&](const int32_t* slots, int c) {
      if constexpr (!FP8) {
        const auto* pool = static_cast<const __nv_bfloat16*>(pages.pool);
        const int v = lane & 7;  // eight lanes to a row's 128 bytes
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int q = k * 16 + rw * 4 + (lane >> 3);
          const int64_t slot = slots[q];
          lat::copy16(smem_u32(a_smem + c % kAhead * kUnit + q * 128 + ((v ^ (q & 7)) << 4)),
                      pool + max(slot, static_cast<int64_t>(0)) * kRow + c * 64 + v * 8,
                      slot >= 0 ? 16u : 0u);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      } else {
        const auto* pool = static_cast<const uint8_t*>(pages.pool);
        const int v = lane & 3;  // four lanes to a row's 64 codes
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t slot = slots[k * 32 + rw * 8 + (lane >> 2)];
          raw[c % kAhead][k] = slot >= 0 ? __ldg(reinterpret_cast<const uint4*>(pool + slot * kRow + c * 64) + v)
                                         : make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    auto convert = [&](int c) {  // FP8: the codes in registers, as bf16 (exact), to shared memory
      const int v = lane & 3;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int q = k * 32 + rw * 8 + (lane >> 2);
        const uint4 x4 = raw[c % kAhead][k];
        const uint32_t cc[4] = {x4.x, x4.y, x4.z, x4.w};
        uint32_t y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 x = lat::e4m3_values(cc[e >> 1] >> (16 * (e & 1)) & 0xFFFFu);
          y[e] = pack_bf16x2(x.x, x.y);
        }
        uint8_t* at = a_smem + c % kAhead * kUnit + q * 128;
        *reinterpret_cast<uint4*>(at + (((2 * v) ^ (q & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(at + (((2 * v + 1) ^ (q & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
      }
    };
    auto start_first = [&](const int32_t* slots) {
#pragma unroll
      for (int c = 0; c < kAhead; ++c) start(slots, c);
    };
    // the rotary part of tile n
    auto rotary = [&](int n) {
      const int64_t row0 = (static_cast<int64_t>(first_tile + n) * kCluster + rank) * kTile;
      for (int i = t; i < kTile * 8; i += kRowThreads) {
        const int q = i >> 3, v = i & 7;
        const int64_t row = row0 + q;
        if (row >= total) break;
        const int64_t slot = ms->slot[n & 1][q];
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (slot >= 0) {
          if (FP8) {
            const uint2 c = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pages.pool) + slot * kRow + LAT) + v);
            const float s = ms->scale[n & 1][q];
            const uint32_t cc[2] = {c.x, c.y};
            float f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 x = lat::e4m3_values(cc[e >> 1] >> (16 * (e & 1)) & 0xFFFFu);
              f[2 * e] = x.x * s;
              f[2 * e + 1] = x.y * s;
            }
            y = lat::pack8(f);
          } else {
            y = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pages.pool) + slot * kRow + LAT) + v);
          }
        }
        reinterpret_cast<uint4*>(k_rope)[row * 8 + v] = y;
      }
    };
    locate(0);
    start_first(ms->slot[0]);
    bool over = false;  // the same in all four warps
    for (int n = 0; n < n_tiles; ++n) {
#pragma unroll
      for (int c = 0; c < C::kChunks; ++c) {
        if constexpr (FP8) {
          convert(c);
          if (c + kAhead < C::kChunks) start(ms->slot[n & 1], c + kAhead);
        } else {
          // all but the chunks after this one have landed, of those asked for so far
          const int later = min(C::kChunks, max(kAhead, c + kAhead - 1)) - c - 1;
          if (later == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
          if (later == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
          if (later == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
          if (later == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        // everybody's part of the chunk is there, and the chunk before has been read (a
        // warp that gives up takes the others along)
        over = lat::bar_any(1, kRowThreads, !ok || *abort_flag != 0);
        if (over) break;
        if (!FP8 && c > 0 && c + kAhead - 1 < C::kChunks) start(ms->slot[n & 1], c + kAhead - 1);
        uint32_t y[32];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const uint4 x = *reinterpret_cast<const uint4*>(a_smem + c % kAhead * kUnit + r * 128 +
                                                          ((v ^ (r & 7)) << 4));
          y[4 * v] = x.x, y[4 * v + 1] = x.y, y[4 * v + 2] = x.z, y[4 * v + 3] = x.w;
        }
        if (n > 0) ok = ok && mbar_wait(&ms->a_empty[c], (n - 1) & 1);
        __syncwarp();
        tc::fence_after();
        tc::st16(tmem + lanes + c * 32, *reinterpret_cast<uint32_t(*)[16]>(&y[0]));
        tc::st16(tmem + lanes + c * 32 + 16, *reinterpret_cast<uint32_t(*)[16]>(&y[16]));
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) lat::arrive_at_first(&ms->a_full[c]);
      }
      // the rows have been read: the next may come
      if (over || (over = lat::bar_any(1, kRowThreads, !ok))) break;
      if (n + 1 < n_tiles) {
        locate(n + 1);
        start_first(ms->slot[(n + 1) & 1]);
      }
      if (n > 0 || first_sub == 0) rotary(n);  // by the CTA that has the tile's first unit
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (over && lane == 0) {
      *abort_flag = 1;
      flag_error(err, PSW_DEVERR_PIPELINE);
    }
  } else if (warp == kWeightWarp) {
    // ------------------------------------------------------------ weights
    const bool one = lat::elect_one();
    int sub = first_sub, box = 0;
    for (int u = 0; ok && u < count; ++u) {
#pragma unroll
      for (int c = 0; c < C::kChunks; c += kBoxChunks, ++box) {
        const int s = box % C::kRing;
        ok = ok && mbar_wait(&ms->w_empty[s], (box / C::kRing & 1u) ^ 1u);
        if (ok && one) {
          mbar_arrive_expect_tx(&ms->w_full[s], kBox);
#pragma unroll
          for (int i = 0; i < kBoxChunks; ++i)
            lat::tma_box(smem_u32(w_ring + s * kBox + i * (kUnit / 2)), &w_map, &ms->w_full[s],
                         (c + i) * 64, sub * kTile + rank * (kTile / kCluster), 0);
        }
      }
      sub = sub + 1 == per_tile ? 0 : sub + 1;
      ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
    }
    if (!ok && one) {
      *abort_flag = 1;
      flag_error(err, PSW_DEVERR_PIPELINE);
      // copies in flight land before the CTAs end
      for (int i = max(0, box - C::kRing); i < box; ++i)
        mbar_wait(&ms->w_full[i % C::kRing], i / C::kRing & 1);
    }
  } else if (warp == kMmaWarp && rank != 0) {
    // ------------------------------------------------------------ second CTA
    // tells the first, which issues the products, what of w has landed here
    const bool one = lat::elect_one();
    const int64_t boxes = static_cast<int64_t>(count) * (C::kChunks / kBoxChunks);
    int s = 0;
    uint32_t phase = 0;
    for (int64_t i = 0; ok && i < boxes; ++i) {
      ok = mbar_wait(&ms->w_full[s], phase);
      if (ok && one) lat::arrive_at_first(&ms->w_full[s]);
      s = s + 1 == C::kRing ? 0 : s + 1;
      phase ^= s == 0 ? 1u : 0u;
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
    constexpr uint32_t id = tc::idesc_bf16_f32(kCluster * kTile, kTile, 0, 0);
    constexpr uint32_t kStep = kBox >> 4;
    const uint64_t w_desc = tc::smem_desc(smem_u32(w_ring), 16, 1024, tc::kSwizzle128B);
    int sub = first_sub, n = 0, s = 0;
    uint32_t phase = 0;
    bool there = false;  // box s has been seen to have landed
    for (int u = 0; ok && u < count; ++u) {
      const bool last = u == count - 1 || sub == per_tile - 1;  // of this tile here
      const bool begins = u == 0 || sub == 0;
      const int acc = u % kAcc;
      ok = mbar_wait(&ms->d_empty[acc], (u / kAcc & 1u) ^ 1u);
      tc::fence_after();
#pragma unroll
      for (int c0 = 0; c0 < C::kChunks; c0 += kBoxChunks) {
        if (!there) ok = ok && mbar_wait(&ms->w_full[s], phase);
        const uint64_t wd = w_desc + s * kStep;
        uint64_t* empty = &ms->w_empty[s];
        s = s + 1 == C::kRing ? 0 : s + 1;
        phase ^= s == 0 ? 1u : 0u;
#pragma unroll
        for (int i = 0; i < kBoxChunks; ++i) {
          const int c = c0 + i;
          if (begins) {
            ok = ok && mbar_wait(&ms->a_full[c], n & 1);
            tc::fence_after();
          }
          if (ok && one) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              lat::mma_ts_pair(tmem + C::kTmemD + acc * kTile, tmem + c * 32 + k * 8,
                               wd + i * (kUnit / 2 >> 4) + k * 2, id, (c > 0 || k > 0) ? 1u : 0u);
            if (last) lat::commit_pair(&ms->a_empty[c]);
          }
          // whether the next box has landed is asked while the products are issued
          if (i == 0) there = mbar_test(&ms->w_full[s], phase);
        }
        if (ok && one) lat::commit_pair(empty);
      }
      if (ok && one) lat::commit_pair(&ms->d_full[acc]);
      if (last) ++n;
      sub = sub + 1 == per_tile ? 0 : sub + 1;
      ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
    }
    if (one) {
      if (!ok) {
        *abort_flag = 1;
        flag_error(err, PSW_DEVERR_PIPELINE);
      }
      lat::commit_pair(&ms->drained);  // every MMA has ended before tensor memory is freed
      mbar_wait(&ms->drained, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ results
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    uint8_t* mine = stage + warp * 2048;
    int sub = first_sub, n = 0;
    for (int u = 0; u < count; ++u) {
      const int acc = u % kAcc, buf = n & 1;
      const bool last = u == count - 1 || sub == per_tile - 1;
      if (FP8 && (u == 0 || sub == 0)) ok = mbar_wait(&ms->rows_set[buf], n >> 1 & 1);
      ok = __all_sync(0xffffffffu, ok && mbar_wait(&ms->d_full[acc], u / kAcc & 1) && *abort_flag == 0);
      if (!ok) break;
      tc::fence_after();
      const float s = FP8 ? ms->scale[buf][warp * 32 + lane] : 1.f;
      const int64_t row0 =
          (static_cast<int64_t>(first_tile + n) * kCluster + rank) * kTile + warp * 32;
      const int head = sub >> 1, part = sub & 1;
#pragma unroll
      for (int g = 0; g < 4; ++g) {  // 32 columns at a time
        uint32_t v[32];
        tc::ld32(tmem + lanes + C::kTmemD + acc * kTile + g * 32, v);
        tc::wait_ld();
        if (g == 3) {  // the accumulator has been read
          tc::fence_before();
          __syncwarp();
          if (lane == 0) lat::arrive_at_first(&ms->d_empty[acc]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = FP8 ? __uint_as_float(v[q * 8 + e]) * s : __uint_as_float(v[q * 8 + e]);
          *reinterpret_cast<uint4*>(mine + lane * 64 + ((q ^ (lane >> 1 & 3)) << 4)) = lat::pack8(y);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = k * 8 + (lane >> 2), q = lane & 3;
          const uint4 y = *reinterpret_cast<const uint4*>(mine + r * 64 + ((q ^ (r >> 1 & 3)) << 4));
          if (row0 + r < total)
            *reinterpret_cast<uint4*>(kv + ((row0 + r) * heads + head) * kLatentKv +
                                      part * kTile + g * 32 + q * 8) = y;
        }
        __syncwarp();
      }
      if (last) {
        if (lane == 0) mbar_arrive(&ms->rows_done[buf]);
        ++n;
      }
      sub = sub + 1 == per_tile ? 0 : sub + 1;
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      flag_error(err, PSW_DEVERR_PIPELINE);
    }
  }
  __syncwarp();
  tc::fence_before();
  lat::cluster_sync();  // nobody leaves while the other may still reach into it
  if (warp == kMmaWarp) lat::dealloc_pair(tmem, 512);
}

template <int LAT, bool FP8>
int launch(const LatentArgs& L, const LatentPages& pages, const int32_t* cu_k,
           const int32_t* k_first, int n_seqs, int n_k_total, const void* w, void* kv,
           void* k_rope, int num_sms, int32_t* err, cudaStream_t stream) {
  using C = Cfg<LAT>;
  CUtensorMap w_map;
  int rc = make_map_3d(&w_map, false, w, {LAT, static_cast<int64_t>(L.n_heads) * kLatentKv, 1},
                       {2 * LAT, 2 * LAT}, {64, kTile / kCluster, 1});
  if (rc != PSW_OK) return rc;
  auto* kernel = latent_expand_kernel<LAT, FP8>;
  rc = set_smem_limit(reinterpret_cast<const void*>(kernel), C::kSmemBytes);
  if (rc != PSW_OK) return rc;
  kernel<<<num_sms / kCluster * kCluster, kThreads, C::kSmemBytes, stream>>>(
      w_map, pages, cu_k, k_first, n_seqs, n_k_total, L.n_heads,
      static_cast<__nv_bfloat16*>(kv), static_cast<__nv_bfloat16*>(k_rope), err);
  return cudaGetLastError() == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

}  // namespace lexp

int launch_latent_expand(const LatentArgs& L, const LatentPages& pages, const int32_t* cu_k,
                         const int32_t* k_first, int n_seqs, int n_k_total, const void* w,
                         void* kv, void* k_rope, int num_sms, int32_t* err, cudaStream_t stream) {
  const bool fp8 = pages.row_scale != nullptr;
  auto* go = L.latent == 512 ? (fp8 ? lexp::launch<512, true> : lexp::launch<512, false>)
                             : (fp8 ? lexp::launch<256, true> : lexp::launch<256, false>);
  return go(L, pages, cu_k, k_first, n_seqs, n_k_total, w, kv, k_rope, num_sms, err, stream);
}

}  // namespace psw
