// fp4_decode.cu -- attention of one token per sequence over 4-bit pages.
//
//   s_j = scale * <q, K_j>, capped;  out = sum_j softmax(s)_j V_j
// over the keys that window and length leave, K_j and V_j being code * block
// scale * tensor scale. One kernel launch.
//
// What bounds it (GPU time of a call, 16-token pages): with K and V in two pools the
// pages' bytes, read at 5.9 of the measured 6.7 TB/s once under way, and about 5 us each
// to begin (lengths, places, queries, first pages) and to end (the slowest warp, joins):
// 3 sequences of 40001 to 65536, 7 KV heads, 60 us for 302 MB; 64 that see 1024
// keys, 8 KV heads, 36 us for 149 MB. Where one page serves as both (k_eq_v) it is
// read once and worked on twice: 32 sequences of 1024 to 32768, head size 512, take 121 us
// for 365 MB, a page 1460 cycles of an SM quarter. 1030 of those are the products and
// the scalings of codes, which share the quarter's half-precision port; the others are latency that
// two warps of 255 registers do not hide (890 instructions a page; for each of them a warp stands 0.94
// cycles at one that it depends on, 0.44 at the port, 0.25 at instructions not fetched yet).
// More than 8 query heads to a KV head are units of their own, which read and convert the pages
// again: 16 sequences of 6000 to 16384, 4 KV heads, take 42.6 us with 8 query heads to each
// and 69.6 with 16, at head size 512 with k_eq_v 68.1 and 121.
//
//  * Every warp of a persistent grid is a worker of its own (list, runs and joins are
//    in fp4_decode.cuh): its own ring of pages in shared memory, filled by plain bulk
//    copies (a page of a head is one run of bytes), its own running maximum, sum and
//    output. No warp waits for another before the joins. Scores and values in warps of
//    their own (head size 512) took 141 us instead of 121, two warps to a unit 151.
//  * A page is 16 keys, the M side of S^T = K Q^T (mma.sync, 16 keys x 16 values x 8
//    heads); the values are the M side of O^T = V^T P^T. With the large operand
//    on the M side a product takes 8 of its values per lane and no operand is
//    padded but by missing heads. Codes become f16 by the hardware's conversion,
//    two at a time; times their block's E4M3 scale they are still exact in f16
//    (2 + 4 significant bits, 2^-10 .. 2688). For V^T the codes of two keys of
//    one value have to be neighbours: they are exchanged as codes, four to a
//    byte operation, before the conversion.
//  * P = 2^(z - m) with m 6 to 14 below the largest score so far (log2 units),
//    rounded once to f16: the result is bf16, half a step of f16 is 1/8 of
//    its. m moves, and O is rescaled, only when a score passes m + 14, so P stays
//    below 2^14 and what lies 30 octaves below the largest is still counted.
//  * q is multiplied by a power of two per head so that its largest value lies in
//    [2^14, 2^15): in f16 all but values 2^-28 of that are exact.
#include <float.h>

#include "fp4_decode.cuh"

namespace psw {
namespace {

using namespace fp4;

template <int HD, bool KEQV>
struct Cfg {
  static constexpr int kWarps = HD == 256 ? 12 : 8;  // registers: 168 and 255 a thread
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kParts = HD / 256;
  static constexpr int kTensors = KEQV ? 1 : 2;
  static constexpr int kTile = HD == 512 && !KEQV ? 1 : 2;  // pages that a warp works on at a time
  static constexpr int kPageBytes = Page<HD>::kBytes * kTensors;
  static constexpr int kTileBytes = kTile * kPageBytes;
  static constexpr int kRingBytes = 18432;  // per warp
  static constexpr int kStages = kRingBytes / kTileBytes;
  // Pages that a CTA could work on while the parts of several are joined: a sequence of 256, 8 KV
  // heads, takes 7.8 us with a CTA for each head and 9.9 cut into equal runs, 19 of 1024 (152
  // units) 17.2 and 19.0, pages from memory. With pages in L2: one of 1024 13.5 and 10.7, 19 of them
  // 13.9 and 15.8. (Head size 512, 4 heads, in L2: 256 11.2 and 12.3, 1024 22.0 and 13.6; k_eq_v 512
  // 14.6 and 14.7, 1024 20.7 and 14.7.)
  static constexpr int kApart = HD == 256 ? 28 : KEQV ? 32 : 18;
  static constexpr int kQBytes = HD == 256 ? 0 : HD * 8 * 2;  // per warp: q as operands (HD 512)
  static constexpr int kSmem = kWarps * (kRingBytes + kQBytes);
  static_assert(kWarps <= kMaxWorkers && 2 * kWarps <= 32, "pieces of a CTA");
  static_assert(kStages * kTileBytes == kRingBytes && kStages >= 2 && kStages <= 8, "ring");
  static_assert(HD * 8 * 4 <= kRingBytes, "a piece's output fits where the ring was");
  static_assert(HD * 8 * 4 + 2 * kWarps * 8 * 4 <= kRingBytes, "and its weights");
  static_assert(3 * kMaxCtas * kMaxJobs * 4 <= PSW_FP4_COUNTER_BYTES && kMaxJobs == 8, "tickets");
};

template <int HD, bool KEQV>
__global__ void __launch_bounds__(Cfg<HD, KEQV>::kThreads, 1) fp4_decode_kernel(const Args a) {
  using C = Cfg<HD, KEQV>;
  constexpr int W = C::kWarps, S = C::kStages, TP = C::kTile;
  constexpr int kUnitCost = fp4_unit_cost(HD);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_full[W][S];
  __shared__ Piece s_piece[2 * W];
  __shared__ float2 s_ml[2 * W][kQHeadsPerUnit];
  __shared__ ListSmem s_list;
  // a warp's unit that is worked on, and that of the next page to fetch: wanted at a unit's
  // ends alone, and no registers are to spare between them
  __shared__ Place s_now[W], s_next[W];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::kRingBytes;
  const int ups = a.n_kv * a.qchunks, hp = a.rows / 2;

  if (lane < S) mbar_init(&s_full[warp][lane], 1);
  fence_mbar_init();
  if (tid < 2 * W) s_piece[tid].pages = 0;
  const Run run = begin_run<W>(a, s_list, warp, kUnitCost, C::kApart);
  const int me = run.me;
  int page = run.page;   // the next page of the unit that is worked on
  int left = run.left;   // entries of the run from the next page to fetch on
  int np = 0;            // pages of the unit
  if (left > 0) {
    np = run.c.s.np;
    if (lane == 0) s_now[warp] = s_next[warp] = run.c;
    __syncwarp();
    // ---- fetching: a tile's blocks, a copy by each of the first lanes
    int f_page = page, f_np = np, ids_at = 0;
    int32_t ids = 0;     // lane i: block of page ids_at + i
    int n = 0;           // tiles asked for
    uint32_t info = 0;   // four bits per stage: more than one page; pages without a valid block
    const int stall = static_cast<int>(blockIdx.x) == a.stall_cta && warp == 0 ? a.stall_tile : -1;
    const int my_page = lane / C::kTensors;  // of a tile (lanes below kTile * kTensors)
    const bool my_v = C::kTensors == 2 && (lane & 1);
    const uint8_t* f_from = nullptr;  // this lane's tensor, at the unit's KV head of block 0
    auto fetch_unit = [&]() {
      const Place& f = s_next[warp];
      f_from = (my_v ? a.v_pool : a.k_pool) +
               static_cast<int64_t>(f.j / a.qchunks) * Page<HD>::kBytes;
    };
    auto fetch_ids = [&]() {
      const Place& f = s_next[warp];
      ids_at = f_page;
      const int at = f_page + lane;
      ids = at < f_np
                ? __ldg(a.table + static_cast<int64_t>(f.b) * a.max_blocks + f.s.p0 + at)
                : 0;
    };
    auto fetch = [&]() {  // the next tile of the run, if there is one
      if (f_page == f_np) {
        left -= kUnitCost;
        if (left <= 0) return;
        const Place f = next_place(&s_next[warp], a, ups, kUnitCost);
        f_np = f.s.np;
        f_page = 0;
        fetch_unit();
        fetch_ids();
        // its queries are wanted when the pages before it are done
        const char* q = reinterpret_cast<const char*>(
            a.q + (static_cast<int64_t>(f.b) * a.n_q + first_head(a, f.j)) * HD);
        for (int k = lane * 128; k < heads_of(a, f.j) * HD * 2; k += 32 * 128)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q + k));
      }
      if (f_page - ids_at > 32 - TP) fetch_ids();
      const int pages = min(min(TP, f_np - f_page), left);
      int32_t blk = __shfl_sync(0xffffffffu, ids, (f_page - ids_at + my_page) & 31);
      const int st = n & (S - 1);
      const bool mine = lane < pages * C::kTensors;
      const bool wrong = mine && static_cast<uint32_t>(blk) >= static_cast<uint32_t>(a.num_blocks);
      uint32_t word = pages > 1 ? 1u : 0u;
      if (const uint32_t no = __ballot_sync(0xffffffffu, wrong)) {  // (a lane of a tensor each)
        if (wrong) blk = 0;
        word |= (no & 1u ? 2u : 0u) | (no >> C::kTensors & 1u ? 4u : 0u);
        if (lane == 0) flag_error(a.err, PSW_DEVERR_BLOCK_ID);
      }
      info = (info & ~(15u << (4 * st))) | word << (4 * st);
      const bool ask = n != stall;
      expect_if(lane == 0 && ask, &s_full[warp][st], pages * C::kPageBytes);
      bulk_load_if(mine && ask, smem_u32(ring + st * C::kTileBytes + lane * Page<HD>::kBytes),
                   f_from + static_cast<int64_t>(blk) * a.page_stride, Page<HD>::kBytes,
                   &s_full[warp][st]);
      f_page += pages;
      left -= pages;
      ++n;
    };

    // tokens of this lane: rows g, g + 8 of S^T are tokens r0, r0 + 8; key slots 2 t, 2 t + 1
    // (and + 8) of P are tokens ra, rb (and + 8). This order keeps both products' loads free of
    // bank conflicts (the pages' units are exchanged by the token's low bits).
    const int r0 = (g & 1) ? (((g & 6) ^ 4) | 1) : g;
    const int ra = 2 * t, rb = ((2 * t) ^ 4) | 1;
    constexpr int kRow = Page<HD>::kScaleRow, kCodes = Page<HD>::kCodeBytes;
    int k_at = r0 * 128 + ((t ^ (r0 & 7)) << 4);  // unit t; unit 4 + t: ^ 64
    int ks_at = kCodes + r0 * kRow + t * Page<HD>::kLaneScales;
    int va_at = ra * 128 + ((g ^ ra) << 4), vb_at = rb * 128 + ((g ^ rb) << 4);
    int vs_at = kCodes + (g & 3) * Page<HD>::kLaneScales + (g >> 2) * (HD / 128) + ra * kRow;
    // (kept in registers: formed anew for every tile they would cost as much as the softmax)
    asm volatile("" : "+r"(k_at), "+r"(ks_at), "+r"(va_at), "+r"(vb_at), "+r"(vs_at));
    const int vs_b = (rb - ra) * kRow;

    uint32_t qr[HD == 256 ? 32 : 1];  // q as operands: HD 256 in registers, HD 512 in shared memory
    uint4* q_smem = reinterpret_cast<uint4*>(smem + W * C::kRingBytes + warp * C::kQBytes) + lane;
    float qf[2];              // factor of the scores of heads 2 t, 2 t + 1
    float acc[HD / 16][4];    // value 32 g + 2 i (+ 256 part): heads 2 t, 2 t + 1; then the next
    float m[2], l[2];
    int piece_from = 0;
    uint32_t ends = 0;  // a bit per token seen of the unit's first page, and of its last
    uint4 raw[HD / 128][4];

    auto load_q = [&]() {
      const Place& c = s_now[warp];
      const int row = first_head(a, c.j) + min(g, heads_of(a, c.j) - 1);
      const uint4* src =
          reinterpret_cast<const uint4*>(a.q + (static_cast<int64_t>(c.b) * a.n_q + row) * HD) +
          t * 4;
#pragma unroll
      for (int k = 0; k < HD / 128; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[k][i] = __ldg(src + k * 16 + i);
    };
    auto begin_piece = [&]() {
      uint32_t top = 0;  // the largest |q|, as bf16 bits
#pragma unroll
      for (int k = 0; k < HD / 128; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w[4] = {raw[k][i].x, raw[k][i].y, raw[k][i].z, raw[k][i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7FFF7FFFu);
        }
      uint32_t big = max(top & 0xFFFFu, top >> 16);
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      const int e = max(static_cast<int>(big >> 7), 15);  // exponent of 2 + 127
      const float up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);   // 2^(141 - e)
      const float down = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);  // 2^(e - 141)
      // (columns of heads that are not there repeat the last one: their results go nowhere)
#pragma unroll
      for (int k = 0; k < HD / 128; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w[4] = {raw[k][i].x, raw[k][i].y, raw[k][i].z, raw[k][i].w};
          uint32_t h[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 v = unpack_bf16x2(w[x]);
            h[x] = pack_f16x2(v.x * up, v.y * up);
            if constexpr (HD == 256) qr[(k * 4 + i) * 4 + x] = h[x];
          }
          if constexpr (HD != 256) q_smem[(k * 4 + i) * 32] = make_uint4(h[0], h[1], h[2], h[3]);
        }
      // (limited: under a cap far below the scores it can pass fp32, and a score of 0 has to stay 0)
      const float fac =
          fminf(a.scale * down * (a.softcap > 0.f ? 1.f / a.softcap : lat::kLog2e), FLT_MAX);
      qf[0] = __shfl_sync(0xffffffffu, fac, 8 * t);
      qf[1] = __shfl_sync(0xffffffffu, fac, 8 * t + 4);
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[i][x] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
      piece_from = page;
      const Place& c = s_now[warp];
      ends = ((0xFFFFu << (c.s.lo & (kBlockSize - 1))) & 0xFFFFu) |
             (0xFFFFu >> (kBlockSize - 1 - ((c.s.len - 1) & (kBlockSize - 1)))) << 16;
    };
    auto sum_l = [&]() {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
        l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
      }
    };
    // this lane's outputs as float4s of the piece
    auto put = [&](float4* dst) {
      if (t >= hp) return;
#pragma unroll
      for (int part = 0; part < C::kParts; ++part)
#pragma unroll
        for (int odd = 0; odd < 2; ++odd)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float(&x)[4] = acc[part * 16 + 2 * i];
            const float(&y)[4] = acc[part * 16 + 2 * i + 1];
            dst[((part * 2 + odd) * 8 + i) * 8 * hp + g * hp + t] =
                make_float4(x[odd], x[2 + odd], y[odd], y[2 + odd]);
          }
    };
    auto note = [&](int at) {  // the piece, for the CTA
      if (g == 0) {
        s_ml[at][2 * t] = make_float2(m[0], l[0]);
        s_ml[at][2 * t + 1] = make_float2(m[1], l[1]);
      }
      const Place& c = s_now[warp];
      if (lane == 0) s_piece[at] = Piece{c.b, c.j, c.tile0, c.s.np, page - piece_from};
    };

    load_q();  // (in front of the pages: behind them it would wait for all)
    fetch_unit();
    fetch_ids();
    for (int i = 0; i < S && left > 0; ++i) fetch();
    begin_piece();
    bool failed = false;
    for (int it = 0; it < n; ++it) {
      const int st = it & (S - 1);
      if (!landed(&s_full[warp][st], (it / S) & 1)) {
        failed = true;
        break;
      }
      const uint8_t* tile = ring + st * C::kTileBytes;
      const uint32_t word = info >> (4 * st);
      const int pages = TP == 1 ? 1 : 1 + (word & 1);
      // a bit per token of the tile: visible
      constexpr uint32_t kAll = TP == 1 ? 0xFFFFu : 0xFFFFFFFFu;
      uint32_t seen = pages == TP ? kAll : 0xFFFFu;
      if (page == 0) seen &= 0xFFFF0000u | ends;
      if (page + pages == np)
        seen &= pages == 1 ? ends >> 16 : (ends & 0xFFFF0000u) | 0xFFFFu;
      const bool edge = seen != kAll || (word & 6) != 0;

      // ---- S^T = K Q^T
      // a page's products in two sums where there are few warps (16 sequences of 6000 to 16384, 4 KV
      // heads, 71.2 -> 69.9 us; k_eq_v, 32 of 1024 to 32768, 122.2 -> 121.2; at HD 256 the registers
      // cost more: 64 of 512 to 4096 36.1 -> 37.0)
      constexpr int kSums = HD == 512 ? 2 : 1;
      float s[TP * kSums][4];
#pragma unroll
      for (int pg = 0; pg < TP * kSums; ++pg)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[pg][x] = 0.f;
      {
        uint32_t ks[TP][2][HD / 256];  // scale bytes of tokens r0, r0 + 8
#pragma unroll
        for (int pg = 0; pg < TP; ++pg)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint8_t* p = tile + pg * C::kPageBytes + ks_at + r * 8 * kRow;
            if constexpr (HD == 256) {
              ks[pg][r][0] = *reinterpret_cast<const uint32_t*>(p);
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(p);
              ks[pg][r][0] = x.x;
              ks[pg][r][1] = x.y;
            }
          }
#pragma unroll
        for (int k = 0; k < HD / 128; ++k) {
          const int place = HD == 256 ? k : 2 * (k & 1) + (k >> 1);  // of the 128 values' scales
          uint4 ka[TP], kb[TP];
          uint32_t ea[TP][2], eb[TP][2];
#pragma unroll
          for (int pg = 0; pg < TP; ++pg) {
            const uint8_t* p =
                tile + pg * C::kPageBytes + (k >> 1) * 2048 + (k_at ^ ((k & 1) * 64));
            ka[pg] = *reinterpret_cast<const uint4*>(p);
            kb[pg] = *reinterpret_cast<const uint4*>(p + 1024);
            const uint32_t sa = fp4::scales_f16(ks[pg][0][place >> 1] >> (16 * (place & 1)));
            const uint32_t sb = fp4::scales_f16(ks[pg][1][place >> 1] >> (16 * (place & 1)));
            ea[pg][0] = __byte_perm(sa, 0, 0x1010);
            ea[pg][1] = __byte_perm(sa, 0, 0x3232);
            eb[pg][0] = __byte_perm(sb, 0, 0x1010);
            eb[pg][1] = __byte_perm(sb, 0, 0x3232);
          }
#pragma unroll
          for (int jp = 0; jp < 4; ++jp) {  // two products, of 4 values each of every lane's unit
            uint4 qq;
            if constexpr (HD == 256)
              qq = make_uint4(qr[k * 16 + jp * 4], qr[k * 16 + jp * 4 + 1], qr[k * 16 + jp * 4 + 2],
                              qr[k * 16 + jp * 4 + 3]);
            else
              qq = q_smem[(k * 4 + jp) * 32];
            const int h = jp >> 1;
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int pg = 0; pg < TP; ++pg) {
                const uint32_t wa = word_at(ka[pg], jp), wb = word_at(kb[pg], jp);
                const uint32_t x[4] = {mul_f16x2(codes_at(wa, 2 * half), ea[pg][h]),
                                       mul_f16x2(codes_at(wb, 2 * half), eb[pg][h]),
                                       mul_f16x2(codes_at(wa, 2 * half + 1), ea[pg][h]),
                                       mul_f16x2(codes_at(wb, 2 * half + 1), eb[pg][h])};
                mma_f16(s[pg * kSums + half % kSums], x, half ? qq.z : qq.x, half ? qq.w : qq.y);
              }
          }
        }
      }
      // ---- softmax: tokens r0, r0 + 8 of heads 2 t, 2 t + 1
      float z[TP][4];
#pragma unroll
      for (int pg = 0; pg < TP; ++pg)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          z[pg][x] = (kSums == 1 ? s[pg][x] : s[pg * kSums][x] + s[pg * kSums + kSums - 1][x]) *
                     qf[x & 1];
      if (a.softcap > 0.f) {
#pragma unroll
        for (int pg = 0; pg < TP; ++pg)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            z[pg][x] = a.softcap * lat::kLog2e * lat::tanh_of(z[pg][x]);
      }
      if (edge) {
#pragma unroll
        for (int pg = 0; pg < TP; ++pg) {
          const uint32_t mask = seen >> (16 * pg);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if ((word >> (1 + pg)) & 1) z[pg][x] = 0.f;
            if (!((mask >> (r0 + (x >> 1) * 8)) & 1)) z[pg][x] = -INFINITY;
          }
        }
      }
      float top[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        top[x] = fmaxf(z[0][x], z[0][2 + x]);
        if (TP == 2) top[x] = max3f(top[x], z[TP - 1][x], z[TP - 1][2 + x]);
      }
      // (m + 14 rounded down: to nearest, it would be m + 16 where m is above 2^25, and P infinite)
      const float lim[2] = {__fadd_rd(m[0], 14.f), __fadd_rd(m[1], 14.f)};
      if (__any_sync(0xffffffffu, top[0] > lim[0] || top[1] > lim[1])) {
        float al[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], o));
          const float mn = top[x] > lim[x] ? top[x] - 6.f : m[x];
          al[x] = m[x] == mn ? 1.f : ex2_approx(m[x] - mn);
          m[x] = mn;
          l[x] *= al[x];
        }
        const uint64_t al2 = f2_pack(al[0], al[1]);
#pragma unroll
        for (int i = 0; i < HD / 16; ++i)
#pragma unroll
          for (int x = 0; x < 4; x += 2) {
            const float2 r = f2_unpack(f2_mul(f2_pack(acc[i][x], acc[i][x + 1]), al2));
            acc[i][x] = r.x;
            acc[i][x + 1] = r.y;
          }
      }
      uint32_t p[TP][2];
#pragma unroll
      for (int pg = 0; pg < TP; ++pg) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          z[pg][x] = ex2_approx(z[pg][x] - m[x & 1]);
          l[x & 1] += z[pg][x];
        }
        p[pg][0] = transposed(pack_f16x2(z[pg][0], z[pg][1]));
        p[pg][1] = transposed(pack_f16x2(z[pg][2], z[pg][3]));
      }

      // ---- O^T += V^T P^T
#pragma unroll
      for (int pg = 0; pg < TP; ++pg) {
        if (pg > 0 && pages == 1) break;
        const uint8_t* vp = tile + pg * C::kPageBytes + (KEQV ? 0 : Page<HD>::kBytes);
        uint32_t vs[4];  // scale bytes of tokens ra, rb, ra + 8, rb + 8: two blocks per part
        const int rows[4] = {ra, rb, ra + 8, rb + 8};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint8_t* x = vp + vs_at + (r & 1 ? vs_b : 0) + (r >> 1) * 8 * kRow;
          if constexpr (HD == 256)
            vs[r] = *reinterpret_cast<const uint16_t*>(x);
          else
            vs[r] = *reinterpret_cast<const uint32_t*>(x);
        }
        if (edge) {  // what rows without a key hold may be anything: 0 times a number
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (((word >> (1 + pg)) & 1) || !((seen >> (16 * pg + rows[r])) & 1)) vs[r] = 0;
        }
#pragma unroll
        for (int part = 0; part < C::kParts; ++part) {
          const uint4 va = *reinterpret_cast<const uint4*>(vp + part * 2048 + va_at);
          const uint4 vb = *reinterpret_cast<const uint4*>(vp + part * 2048 + vb_at);
          const uint4 vc = *reinterpret_cast<const uint4*>(vp + part * 2048 + va_at + 1024);
          const uint4 vd = *reinterpret_cast<const uint4*>(vp + part * 2048 + vb_at + 1024);
          const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
          const uint32_t wc[4] = {vc.x, vc.y, vc.z, vc.w}, wd[4] = {vd.x, vd.y, vd.z, vd.w};
          const uint32_t b01 = __byte_perm(vs[0], vs[1], part == 0 ? 0x5140 : 0x7362);
          const uint32_t b89 = __byte_perm(vs[2], vs[3], part == 0 ? 0x5140 : 0x7362);
          const uint32_t e01[2] = {fp4::scales_f16(b01), fp4::scales_f16(b01 >> 16)};
          const uint32_t e89[2] = {fp4::scales_f16(b89), fp4::scales_f16(b89 >> 16)};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            constexpr uint32_t kLow = 0x0F0F0F0Fu;
            // bytes of (first key, second key) of the even and of the odd values of a word
            const uint32_t lo01 = select_bits(kLow, wa[w], wb[w] << 4);
            const uint32_t hi01 = select_bits(kLow, wa[w] >> 4, wb[w]);
            const uint32_t lo89 = select_bits(kLow, wc[w], wd[w] << 4);
            const uint32_t hi89 = select_bits(kLow, wc[w] >> 4, wd[w]);
            const uint32_t f01 = e01[w >> 1], f89 = e89[w >> 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t x[4] = {
                  mul_f16x2(codes_at(lo01, i), f01), mul_f16x2(codes_at(hi01, i), f01),
                  mul_f16x2(codes_at(lo89, i), f89), mul_f16x2(codes_at(hi89, i), f89)};
              mma_f16(acc[part * 16 + w * 4 + i], x, p[pg][0], p[pg][1]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the tile
      if (left > 0) fetch();
      page += pages;
      if (page == np && it + 1 < n) {  // the unit ends and the run goes on
        sum_l();
        if (page - piece_from == np) {
          const Place& c = s_now[warp];
          const int nh = heads_of(a, c.j), h0 = first_head(a, c.j);
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            if (2 * t + odd >= nh) continue;
            const float fo = a.v_scale / l[odd];
            uint4* dst = reinterpret_cast<uint4*>(
                a.out + (static_cast<int64_t>(c.b) * a.n_q + h0 + 2 * t + odd) * HD + 32 * g);
#pragma unroll
            for (int part = 0; part < C::kParts; ++part)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const float(&o)[4] = acc[part * 16 + 4 * i + x];
                  w[x] = pack_bf16x2(o[odd] * fo, o[2 + odd] * fo);
                }
                dst[part * 32 + i] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            if (g == 0) write_lse(a, Piece{c.b, c.j, 0, 0, 0}, 2 * t + odd, m[odd], l[odd]);
          }
        } else {
          put(a.ws_o + static_cast<int64_t>(me) * (C::kParts * 128 * hp));
          note(2 * warp);
        }
        np = next_place(&s_now[warp], a, ups, kUnitCost).s.np;
        page = 0;
        load_q();
        begin_piece();
      }
    }
    if (failed) {
      if (lane == 0) flag_error(a.err, PSW_DEVERR_PIPELINE);
      for (int i = 0; i < S; ++i) {  // copies in flight have to land: a stage's last phase
        const int last = n - 1 - ((n - 1 - i) & (S - 1));
        if (last >= 0) mbar_wait(&s_full[warp][i], (last / S) & 1);
      }
    } else {
      sum_l();
      put(reinterpret_cast<float4*>(ring));
      note(2 * warp + 1);
    }
  }
  __syncthreads();

  join_pieces<HD, W, W, C::kRingBytes>(a, run.cut, kUnitCost, s_piece, s_ml, smem,
                                       reinterpret_cast<float*>(ring + HD * 8 * 4));
  finish_empty<HD>(a);
}

template <int HD, bool KEQV>
int launch(const Args& a, int num_sms, cudaStream_t stream) {
  using C = Cfg<HD, KEQV>;
  auto* fn = fp4_decode_kernel<HD, KEQV>;
  const int rc = set_smem_limit(reinterpret_cast<const void*>(fn), C::kSmem);
  if (rc != PSW_OK) return rc;
  const int grid = min(num_sms, kMaxCtas);
  fn<<<grid, C::kThreads, C::kSmem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

int slot_rows(const LayerArgs& L) {
  const int heads = L.group() < kQHeadsPerUnit ? L.group() : kQHeadsPerUnit;
  return (heads + 1) / 2 * 2;
}

// Slots of a call: one for every worker's first piece, then those of the CTAs' parts of
// units (CTA + unit: the units of neighbouring CTAs are neighbours, so no two share one).
size_t slots_of(const LayerArgs& L, int n_seqs) {
  return kMaxCtas * (kMaxWorkers + 1) + static_cast<size_t>(n_seqs) * L.n_kv * L.qchunks();
}

}  // namespace

size_t fp4_decode_workspace(const LayerArgs& L, int n_seqs) {
  return kFp4CounterBytes + slots_of(L, n_seqs) * slot_rows(L) * (L.hd * 4 + kMaxJobs * 8);
}

int launch_fp4_decode(const LayerArgs& L, const void* q, const void* k_pool, const void* v_pool,
                      const psw_pages_t& pages, const int32_t* seq_lens, int n_seqs, void* out,
                      float* lse, void* ws, float k_scale, float v_scale, int num_sms,
                      int32_t* err, cudaStream_t stream) {
  Args a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_pool = static_cast<const uint8_t*>(k_pool);
  a.v_pool = static_cast<const uint8_t*>(v_pool);
  a.table = pages.block_table;
  a.seq_lens = seq_lens;
  a.max_blocks = pages.max_blocks_per_seq;
  a.num_blocks = static_cast<int>(pages.num_blocks);
  a.page_stride = static_cast<uint32_t>(L.n_kv) * PSW_FP4_PAGE_BYTES(L.hd);
  a.n_seqs = n_seqs;
  a.n_q = L.n_q;
  a.n_kv = L.n_kv;
  a.group = L.group();
  a.qchunks = L.qchunks();
  a.window = L.window;
  a.scale = L.scale * k_scale;
  // (beyond these fp32 cannot tell a cap from none, or from one that leaves every score 0)
  a.softcap = L.softcap == 0.f ? 0.f : fminf(fmaxf(L.softcap, 0x1p-100f), 0x1p100f);
  a.v_scale = L.k_eq_v ? k_scale : v_scale;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.rows = slot_rows(L);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.tickets = reinterpret_cast<int32_t*>(w);
  a.ws_o = reinterpret_cast<float4*>(w + kFp4CounterBytes);
  a.ws_ml = reinterpret_cast<float2*>(w + kFp4CounterBytes +
                                      slots_of(L, n_seqs) * a.rows * L.hd * 4);
  a.err = err;
  const StallHook hook = stall_hook(kStallDecode);
  a.stall_cta = hook.cta;
  a.stall_tile = hook.tile;
  if (L.hd == 256)
    return L.k_eq_v ? launch<256, true>(a, num_sms, stream)
                    : launch<256, false>(a, num_sms, stream);
  return L.k_eq_v ? launch<512, true>(a, num_sms, stream) : launch<512, false>(a, num_sms, stream);
}

}  // namespace psw
