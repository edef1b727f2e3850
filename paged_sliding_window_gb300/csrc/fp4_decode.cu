// fp4_decode.cu -- attention of one token per sequence over 4-bit pages.
//
//   s_j = scale * <q, K_j>, capped;  out = sum_j softmax(s)_j V_j
// over the keys that window and length leave, K_j and V_j being code * block
// scale * tensor scale. One kernel launch, bound by the pages' bytes where
// K and V are two pools, and by the conversion of codes next to that where one
// page serves as both (k_eq_v).
//
//  * Unit = (sequence, KV head, up to 8 query heads). The visible pages of all
//    units form one list; every warp of a persistent grid (one CTA per SM) is a
//    worker of its own with an equal run of it: its own ring of pages in shared
//    memory, filled by plain bulk copies (a page of a head is one run of bytes),
//    its own running maximum, sum and output. No warp waits for another.
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
//  * A worker's pieces: units that lie in its run alone are written out. The last
//    piece of every warp meets those of the CTA's other warps in shared memory;
//    what is left of a unit goes to the workspace, and whoever adds the
//    unit's last pages (a ticket counts them) joins its pieces, in their order.
#include "fp4.cuh"
#include "latent.cuh"

namespace psw {
namespace {

using fp4::Page;

template <int HD, bool KEQV>
struct Cfg {
  static constexpr int kWarps = HD == 256 ? 12 : 8;  // registers: 168 and 255 a thread
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kParts = HD / 256;
  static constexpr int kChunks = HD / 128;
  static constexpr int kStageBytes = Page<HD>::kBytes * (KEQV ? 1 : 2);
  static constexpr int kRingBytes = 18432;  // per warp: 8, 4 or 2 stages
  static constexpr int kStages = kRingBytes / kStageBytes;
  static constexpr int kQBytes = HD == 256 ? 0 : HD * 8 * 2;  // per warp: q as operands (HD 512)
  static constexpr int kSmem = kWarps * (kRingBytes + kQBytes);
  static_assert(kStages * kStageBytes == kRingBytes, "ring");
  static_assert(HD * 8 * 4 <= kRingBytes, "a piece's output fits where the ring was");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// i is a constant where this is used
__device__ __forceinline__ uint32_t codes_at(uint32_t w, int i) {
  return i == 0 ? fp4::codes_f16<0>(w)
         : i == 1 ? fp4::codes_f16<1>(w)
         : i == 2 ? fp4::codes_f16<2>(w)
                  : fp4::codes_f16<3>(w);
}
// bits of a where m has ones, of b elsewhere
__device__ __forceinline__ uint32_t select_bits(uint32_t m, uint32_t a, uint32_t b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(d) : "r"(m), "r"(a), "r"(b));
  return d;
}

struct Args {
  const __nv_bfloat16* q;
  const uint8_t *k_pool, *v_pool;
  const int32_t *table, *seq_lens;
  int max_blocks;
  int64_t num_blocks;
  int n_seqs, n_q, n_kv, group, qchunks, window;
  float scale, softcap;  // scale: the layer's times K's tensor scale
  float v_scale;
  __nv_bfloat16* out;
  float* lse;
  float4* ws_o;      // [slot][half of a row's pairs ...], see piece_unit
  float2* ws_ml;     // [slot][rows]
  int32_t* tickets;  // [worker]
  int rows;          // rows of a slot: the group's heads, 8 at most, made even
  int32_t* err;
  int stall_cta, stall_tile;
};

struct Seq {
  int len, p0, np, lo;
};
__device__ __forceinline__ Seq seq_of(const Args& a, int b) {
  int len = __ldg(a.seq_lens + b);
  const int cap = a.max_blocks * kBlockSize;
  len = len < 0 ? 0 : (len > cap ? cap : len);
  const int lo = a.window > 0 && len > a.window ? len - a.window : 0;
  const fp4::SeqPages s = fp4::seq_pages(len, lo);
  return Seq{len, s.p0, s.np, lo};
}

// A place in the list of pages: sequence, unit of it, page of the unit.
struct Cursor {
  int b, j, page, tile0;  // tile0: the list's index of the unit's first page
  Seq s;
  __device__ void next_unit(const Args& a, int ups) {
    page = 0;
    tile0 += s.np;
    if (++j < ups) return;
    j = 0;
    do {
      s = seq_of(a, ++b);
    } while (s.np == 0);  // (only called where the list goes on)
  }
};

// What a piece is to the others: its unit and how many of the unit's pages it has.
struct Piece {
  int b, j, tile0, np, pages;
};

// ---- outputs of a piece: float4 number ((part * 2 + odd) * 8 + i) * 8 hp + g hp + t
// holds values 256 part + 32 g + 4 i .. + 3 of head 2 t + odd (hp pairs of heads):
// lane (g, t) of a warp holds 32 neighbouring values of two heads per part.
struct Unit4 {
  int head, d;
};
__device__ __forceinline__ Unit4 piece_unit(int x, int hp) {
  const int t = x % hp, r = x / hp;
  const int g = r & 7, i = (r >> 3) & 7, odd = (r >> 6) & 1, part = r >> 7;
  return Unit4{2 * t + odd, 256 * part + 32 * g + 4 * i};
}

template <int HD>
__device__ __forceinline__ void write_out(const Args& a, const Piece& p, int nh, const Unit4& u,
                                          const float4& o, float inv) {
  if (u.head >= nh) return;
  const int kv = p.j / a.qchunks, h0 = kv * a.group + p.j % a.qchunks * kQHeadsPerUnit;
  __nv_bfloat16* dst = a.out + (static_cast<int64_t>(p.b) * a.n_q + h0 + u.head) * HD + u.d;
  const float f = inv * a.v_scale;
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
}
__device__ __forceinline__ void write_lse(const Args& a, const Piece& p, int head, float m,
                                          float l) {
  const int kv = p.j / a.qchunks, h0 = kv * a.group + p.j % a.qchunks * kQHeadsPerUnit;
  if (a.lse != nullptr)
    a.lse[static_cast<int64_t>(p.b) * a.n_q + h0 + head] = (m + log2f(l)) * lat::kLn2;
}
__device__ __forceinline__ int heads_of(const Args& a, int j) {
  return min(kQHeadsPerUnit, a.group - j % a.qchunks * kQHeadsPerUnit);
}

// The worker that has entry x of a list of `tiles` pages cut for `workers`.
__device__ __forceinline__ int worker_of(int x, int tiles, int workers) {
  return static_cast<int>(((static_cast<int64_t>(x) + 1) * workers - 1) / tiles);
}
__device__ __forceinline__ int run_begin(int w, int tiles, int workers) {
  return static_cast<int>(static_cast<int64_t>(w) * tiles / workers);
}

// Joins all pieces of a unit from the workspace: M = max m_i, l = sum l_i 2^(m_i - M),
// out = sum O_i 2^(m_i - M) / l. There is one piece per CTA (of the unit's first warp there),
// and one more if the last worker's run goes on behind the unit.
template <int HD, bool KEQV>
__device__ void join(const Args& a, const Piece& p, int tiles, int workers, int tid, int threads) {
  constexpr int W = Cfg<HD, KEQV>::kWarps;
  const int ups = a.n_kv * a.qchunks, u = p.b * ups + p.j, nh = heads_of(a, p.j);
  const int hp = a.rows / 2, units = HD / 256 * 128 * hp;
  const int wf = worker_of(p.tile0, tiles, workers);
  const int wl = worker_of(p.tile0 + p.np - 1, tiles, workers);
  const int cf = wf / W, cl = wl / W;
  const bool extra =
      run_begin(wl + 1, tiles, workers) > p.tile0 + p.np && max(wf, cl * W) < wl;
  const int n = cl - cf + 1 + (extra ? 1 : 0);
  auto slot = [&](int i) {
    const int c = cf + i;
    return static_cast<int64_t>(c > cl ? wl : max(wf, c * W)) + u;
  };
  for (int x = tid; x < units; x += threads) {
    const Unit4 q = piece_unit(x, hp);
    if (q.head >= nh) continue;
    float M = -INFINITY, l = 0.f;
    for (int i = 0; i < n; ++i) M = fmaxf(M, __ldcg(&a.ws_ml[slot(i) * a.rows + q.head]).x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const int64_t s = slot(i);
      const float2 ml = __ldcg(&a.ws_ml[s * a.rows + q.head]);
      const float4 v = __ldcg(&a.ws_o[s * units + x]);
      const float f = exp2f(ml.x - M);
      l += ml.y * f;
      o.x += v.x * f;
      o.y += v.y * f;
      o.z += v.z * f;
      o.w += v.w * f;
    }
    write_out<HD>(a, p, nh, q, o, 1.f / l);
    if (q.d == 0) write_lse(a, p, q.head, M, l);
  }
}

template <int HD, bool KEQV>
__global__ void __launch_bounds__(Cfg<HD, KEQV>::kThreads, 1)
fp4_decode_kernel(const Args a) {
  using C = Cfg<HD, KEQV>;
  constexpr int W = C::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_full[W][C::kStages];
  __shared__ int s_run[C::kThreads + 1];
  __shared__ int s_sum[W];
  __shared__ Piece s_piece[W];
  __shared__ float2 s_ml[W][kQHeadsPerUnit];
  __shared__ int s_last[W];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::kRingBytes;
  const int ups = a.n_kv * a.qchunks, hp = a.rows / 2;

  // ---- the list: pages of the sequences before each thread's run of them
  if (lane < C::kStages) mbar_init(&s_full[warp][lane], 1);
  fence_mbar_init();
  const int per = (a.n_seqs + C::kThreads - 1) / C::kThreads;
  int mine = 0;
  for (int b = tid * per; b < min(a.n_seqs, (tid + 1) * per); ++b) mine += seq_of(a, b).np;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_sum[warp] = incl;
  if (lane == 0) s_piece[warp].pages = 0;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < W; ++i) {
    if (i < warp) before += s_sum[i];
    all += s_sum[i];
  }
  s_run[tid + 1] = before + incl;
  if (tid == 0) s_run[0] = 0;
  __syncthreads();
  const int tiles = all * ups;
  const int workers = min(static_cast<int>(gridDim.x) * W, tiles);
  const int me = blockIdx.x * W + warp;

  bool failed = false;
  if (me < workers) {
    const int begin = run_begin(me, tiles, workers);
    const int n = run_begin(me + 1, tiles, workers) - begin;
    Cursor c;  // of the page that is worked on
    {
      const int page = begin / ups;  // units of a sequence are equal: find its sequence by pages
      int lo = 0, hi = C::kThreads;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_run[mid] <= page) lo = mid; else hi = mid;
      }
      c.b = lo * per;
      int off = s_run[lo];
      c.s = seq_of(a, c.b);
      while (page >= off + c.s.np) {
        off += c.s.np;
        c.s = seq_of(a, ++c.b);
      }
      const int rem = begin - off * ups;
      c.j = rem / c.s.np;
      c.page = rem - c.j * c.s.np;
      c.tile0 = begin - c.page;
    }
    Cursor f = c;  // of the next page to fetch
    int fetched = 0, ids_at = 0;
    int32_t ids = 0;
    uint32_t bad = 0;  // a bit per stage: its page has no valid block
    bool ids_ok = false;
    auto fetch = [&]() {
      if (f.page == f.s.np) {
        f.next_unit(a, ups);
        ids_ok = false;
      }
      if (!ids_ok || f.page - ids_at >= 32) {
        ids_at = f.page;
        ids_ok = true;
        ids = f.page + lane < f.s.np
                  ? __ldg(a.table + static_cast<int64_t>(f.b) * a.max_blocks + f.s.p0 + f.page + lane)
                  : 0;
      }
      int32_t blk = __shfl_sync(0xffffffffu, ids, f.page - ids_at);
      const int st = fetched % C::kStages;
      bad &= ~(1u << st);
      if (blk < 0 || blk >= a.num_blocks) {
        bad |= 1u << st;
        if (lane == 0) flag_error(a.err, PSW_DEVERR_BLOCK_ID);
        blk = 0;
      }
      if (lane == 0 && !(static_cast<int>(blockIdx.x) == a.stall_cta && warp == 0 &&
                         fetched == a.stall_tile)) {
        const int64_t at =
            (static_cast<int64_t>(blk) * a.n_kv + f.j / a.qchunks) * Page<HD>::kBytes;
        const uint32_t dst = smem_u32(ring + st * C::kStageBytes);
        mbar_arrive_expect_tx(&s_full[warp][st], C::kStageBytes);
        lat::bulk_load(dst, a.k_pool + at, Page<HD>::kBytes, &s_full[warp][st]);
        if (!KEQV)
          lat::bulk_load(dst + Page<HD>::kBytes, a.v_pool + at, Page<HD>::kBytes,
                         &s_full[warp][st]);
      }
      ++f.page;
      ++fetched;
    };
    for (int i = 0; i < min(n, C::kStages); ++i) fetch();

    // tokens of this lane: rows g, g + 8 of S^T are tokens r0, r0 + 8; key slots 2 t, 2 t + 1
    // (and + 8) of P are tokens ra, rb (and + 8). This order keeps both products' loads free of
    // bank conflicts (the pages' units are exchanged by the token's low bits).
    const int r0 = (g & 1) ? (((g & 6) ^ 4) | 1) : g;
    const int ra = 2 * t, rb = ((2 * t) ^ 4) | 1;
    const int k_at = r0 * 128 + ((t ^ (r0 & 7)) << 4);  // unit t; unit 4 + t: ^ 64
    const int ks_at = Page<HD>::kCodeBytes + r0 * Page<HD>::kScaleRow + t * Page<HD>::kLaneScales;
    const int va_at = ra * 128 + ((g ^ ra) << 4), vb_at = rb * 128 + ((g ^ rb) << 4);
    const int vs_at = Page<HD>::kCodeBytes + (g & 3) * Page<HD>::kLaneScales + (g >> 2) * (HD / 128);

    uint32_t qr[HD == 256 ? 32 : 1];  // q as operands: HD 256 in registers, HD 512 in shared memory
    uint4* q_smem = reinterpret_cast<uint4*>(smem + W * C::kRingBytes + warp * C::kQBytes) + lane;
    float qf[2];              // factor of the scores of heads 2 t, 2 t + 1
    float acc[HD / 16][4];    // value 32 g + 2 i (+ 256 part): heads 2 t, 2 t + 1; the next value: same
    float m[2], l[2];
    bool open = false;
    int piece_from = 0;

    auto begin_piece = [&]() {
      const int nh = heads_of(a, c.j);
      const int kv = c.j / a.qchunks, h0 = kv * a.group + c.j % a.qchunks * kQHeadsPerUnit;
      const uint4* src = reinterpret_cast<const uint4*>(
                             a.q + (static_cast<int64_t>(c.b) * a.n_q + h0 + min(g, nh - 1)) * HD) +
                         t * 4;
      uint4 raw[C::kChunks][4];
#pragma unroll
      for (int k = 0; k < C::kChunks; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[k][i] = __ldg(src + k * 16 + i);
      uint32_t top = 0;  // the largest |q|, as bf16 bits
#pragma unroll
      for (int k = 0; k < C::kChunks; ++k)
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
      const float up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);    // 2^(141 - e)
      const float down = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);   // 2^(e - 141)
      const bool live = g < nh;
      uint32_t pk[HD == 256 ? 1 : 4];
#pragma unroll
      for (int k = 0; k < C::kChunks; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w[4] = {raw[k][i].x, raw[k][i].y, raw[k][i].z, raw[k][i].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 v = unpack_bf16x2(w[x]);
            const uint32_t h = live ? pack_f16x2(v.x * up, v.y * up) : 0u;
            if constexpr (HD == 256) qr[(k * 4 + i) * 4 + x] = h; else pk[x] = h;
          }
          if constexpr (HD != 256) q_smem[(k * 4 + i) * 32] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      const float fac = a.scale * down * (a.softcap > 0.f ? 1.f / a.softcap : lat::kLog2e);
      qf[0] = __shfl_sync(0xffffffffu, fac, 8 * t);
      qf[1] = __shfl_sync(0xffffffffu, fac, 8 * t + 4);
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[i][x] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
      open = true;
      piece_from = c.page;
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

    for (int it = 0; it < n; ++it) {
      if (c.page == c.s.np) c.next_unit(a, ups);
      if (!open) begin_piece();
      const int st = it % C::kStages;
      if (!mbar_wait(&s_full[warp][st], (it / C::kStages) & 1)) {
        failed = true;
        break;
      }
      const uint8_t* page = ring + st * C::kStageBytes;
      const bool is_bad = (bad >> st) & 1;
      const int pos0 = (c.s.p0 + c.page) * kBlockSize;
      uint32_t seen = 0xFFFFu;  // a bit per token: visible
      if (c.s.len - pos0 < kBlockSize) seen &= (1u << (c.s.len - pos0)) - 1u;
      if (c.s.lo > pos0) seen &= 0xFFFFu << (c.s.lo - pos0);

      // ---- S^T = K Q^T
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      {
        uint32_t ks[2][C::kChunks / 2];  // scale bytes of tokens r0, r0 + 8: two blocks per chunk
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t* p = page + ks_at + r * 8 * Page<HD>::kScaleRow;
          if constexpr (HD == 256) {
            ks[r][0] = *reinterpret_cast<const uint32_t*>(p);
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            ks[r][0] = x.x;
            ks[r][1] = x.y;
          }
        }
#pragma unroll
        for (int k = 0; k < C::kChunks; ++k) {
          const uint8_t* p = page + (k >> 1) * 2048 + (k_at ^ ((k & 1) * 64));
          const uint4 ka = *reinterpret_cast<const uint4*>(p);
          const uint4 kb = *reinterpret_cast<const uint4*>(p + 1024);
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
          const int place = HD == 256 ? k : 2 * (k & 1) + (k >> 1);  // of the chunk's scales
          const uint32_t sa = fp4::scales_f16(ks[0][place >> 1] >> (16 * (place & 1)));
          const uint32_t sb = fp4::scales_f16(ks[1][place >> 1] >> (16 * (place & 1)));
          const uint32_t ea[2] = {__byte_perm(sa, 0, 0x1010), __byte_perm(sa, 0, 0x3232)};
          const uint32_t eb[2] = {__byte_perm(sb, 0, 0x1010), __byte_perm(sb, 0, 0x3232)};
#pragma unroll
          for (int jp = 0; jp < 4; ++jp) {  // two products: 4 values each of 32 lanes' units
            uint4 qq;
            if constexpr (HD == 256)
              qq = make_uint4(qr[k * 16 + jp * 4], qr[k * 16 + jp * 4 + 1], qr[k * 16 + jp * 4 + 2],
                              qr[k * 16 + jp * 4 + 3]);
            else
              qq = q_smem[(k * 4 + jp) * 32];
            const int h = jp >> 1;
            const uint32_t x0[4] = {mul_f16x2(codes_at(wa[jp], 0), ea[h]),
                                    mul_f16x2(codes_at(wb[jp], 0), eb[h]),
                                    mul_f16x2(codes_at(wa[jp], 1), ea[h]),
                                    mul_f16x2(codes_at(wb[jp], 1), eb[h])};
            mma_f16(s0, x0, qq.x, qq.y);
            const uint32_t x1[4] = {mul_f16x2(codes_at(wa[jp], 2), ea[h]),
                                    mul_f16x2(codes_at(wb[jp], 2), eb[h]),
                                    mul_f16x2(codes_at(wa[jp], 3), ea[h]),
                                    mul_f16x2(codes_at(wb[jp], 3), eb[h])};
            mma_f16(s1, x1, qq.z, qq.w);
          }
        }
      }
      // ---- softmax: tokens r0, r0 + 8 of heads 2 t, 2 t + 1
      float z[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        z[x] = (is_bad ? 0.f : s0[x] + s1[x]) * qf[x & 1];
        if (a.softcap > 0.f) z[x] = a.softcap * lat::kLog2e * lat::tanh_of(z[x]);
      }
      if (seen != 0xFFFFu) {
        if (!((seen >> r0) & 1)) z[0] = z[1] = -INFINITY;
        if (!((seen >> (r0 + 8)) & 1)) z[2] = z[3] = -INFINITY;
      }
      float top[2] = {fmaxf(z[0], z[2]), fmaxf(z[1], z[3])};
      if (__any_sync(0xffffffffu, top[0] > m[0] + 14.f || top[1] > m[1] + 14.f)) {
        float al[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], o));
          const float mn = top[x] > m[x] + 14.f ? top[x] - 6.f : m[x];
          al[x] = m[x] == mn ? 1.f : ex2_approx(m[x] - mn);
          m[x] = mn;
          l[x] *= al[x];
        }
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          acc[i][0] *= al[0];
          acc[i][1] *= al[1];
          acc[i][2] *= al[0];
          acc[i][3] *= al[1];
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        z[x] = ex2_approx(z[x] - m[x & 1]);
        l[x & 1] += z[x];
      }
      const uint32_t p0 = transposed(pack_f16x2(z[0], z[1]));
      const uint32_t p1 = transposed(pack_f16x2(z[2], z[3]));

      // ---- O^T += V^T P^T
      {
        const uint8_t* vp = page + (KEQV ? 0 : Page<HD>::kBytes);
        uint32_t vs[4];  // scale bytes of tokens ra, rb, ra + 8, rb + 8: two blocks per part
        const int rows[4] = {ra, rb, ra + 8, rb + 8};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint8_t* p = vp + vs_at + rows[r] * Page<HD>::kScaleRow;
          if constexpr (HD == 256)
            vs[r] = *reinterpret_cast<const uint16_t*>(p);
          else
            vs[r] = *reinterpret_cast<const uint32_t*>(p);
        }
        if (seen != 0xFFFFu || is_bad) {  // what these rows hold may be anything: 0 times a number
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (is_bad || !((seen >> rows[r]) & 1)) vs[r] = 0;
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
              mma_f16(acc[part * 16 + w * 4 + i], x, p0, p1);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (fetched < n) fetch();
      ++c.page;
      if (c.page == c.s.np && it + 1 < n) {  // the unit ends and the run goes on
        const Piece p{c.b, c.j, c.tile0, c.s.np, c.page - piece_from};
        sum_l();
        const int nh = heads_of(a, c.j);
        if (p.pages == p.np) {
          const float inv[2] = {1.f / l[0], 1.f / l[1]};
          const int kv = c.j / a.qchunks, h0 = kv * a.group + c.j % a.qchunks * kQHeadsPerUnit;
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            if (2 * t + odd >= nh) continue;
            const float fo = inv[odd] * a.v_scale;
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
            if (g == 0) write_lse(a, p, 2 * t + odd, m[odd], l[odd]);
          }
        } else {
          const int64_t slot = static_cast<int64_t>(me) + c.b * ups + c.j;
          put(a.ws_o + slot * (C::kParts * 128 * hp));
          if (g == 0 && t < hp) {
            a.ws_ml[slot * a.rows + 2 * t] = make_float2(m[0], l[0]);
            a.ws_ml[slot * a.rows + 2 * t + 1] = make_float2(m[1], l[1]);
          }
          __threadfence();
          __syncwarp();
          int last = 0;
          if (lane == 0) {
            int32_t* ticket = a.tickets + worker_of(p.tile0, tiles, workers);
            last = atomicAdd(ticket, p.pages) + p.pages == p.np;
            if (last) *ticket = 0;
          }
          if (__shfl_sync(0xffffffffu, last, 0)) {
            __threadfence();
            join<HD, KEQV>(a, p, tiles, workers, lane, 32);
          }
        }
        open = false;
      }
    }
    if (failed) {  // give up, but not before the copies in flight have landed
      if (lane == 0) flag_error(a.err, PSW_DEVERR_PIPELINE);
      const int at = c.tile0 + c.page - begin;
      for (int i = at + 1; i < fetched; ++i)
        mbar_wait(&s_full[warp][i % C::kStages], (i / C::kStages) & 1);
    } else {
      sum_l();
      put(reinterpret_cast<float4*>(ring));
      if (g == 0) {
        s_ml[warp][2 * t] = make_float2(m[0], l[0]);
        s_ml[warp][2 * t + 1] = make_float2(m[1], l[1]);
      }
      if (lane == 0) s_piece[warp] = Piece{c.b, c.j, c.tile0, c.s.np, c.page - piece_from};
    }
  }
  __syncthreads();

  // ---- the warps' last pieces: runs of warps that share a unit
  const int units = C::kParts * 128 * hp;
  auto first_of_run = [&](int w) {
    return s_piece[w].pages > 0 &&
           (w == 0 || s_piece[w - 1].pages == 0 || s_piece[w - 1].tile0 != s_piece[w].tile0);
  };
  auto run_end = [&](int w, int& pages) {
    int e = w;
    pages = 0;
    for (; e < W && s_piece[e].pages > 0 && s_piece[e].tile0 == s_piece[w].tile0; ++e)
      pages += s_piece[e].pages;
    return e;
  };
  bool cut = false;  // some run is not its whole unit
  for (int w = 0; w < W; ++w) {
    if (!first_of_run(w)) continue;
    const Piece p = s_piece[w];
    int pages;
    const int e = run_end(w, pages);
    const bool whole = pages == p.np;
    cut |= !whole;
    const int nh = heads_of(a, p.j);
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * W + w + p.b * ups + p.j;
    for (int x = tid; x < units; x += C::kThreads) {
      const Unit4 u = piece_unit(x, hp);
      if (u.head >= nh) continue;
      float M = -INFINITY, L = 0.f;
      for (int i = w; i < e; ++i) M = fmaxf(M, s_ml[i][u.head].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = w; i < e; ++i) {
        const float2 ml = s_ml[i][u.head];
        const float4 v = reinterpret_cast<const float4*>(smem + i * C::kRingBytes)[x];
        const float fo = exp2f(ml.x - M);
        L += ml.y * fo;
        o.x += v.x * fo;
        o.y += v.y * fo;
        o.z += v.z * fo;
        o.w += v.w * fo;
      }
      if (whole) {
        write_out<HD>(a, p, nh, u, o, 1.f / L);
        if (u.d == 0) write_lse(a, p, u.head, M, L);
      } else {
        a.ws_o[slot * units + x] = o;
        if (u.d == 0) a.ws_ml[slot * a.rows + u.head] = make_float2(M, L);
      }
    }
  }
  if (cut) {  // (the same for all threads)
    __threadfence();
    __syncthreads();
    if (tid < W) {
      int last = 0;
      if (first_of_run(tid)) {
        const Piece p = s_piece[tid];
        int pages;
        run_end(tid, pages);
        if (pages != p.np) {
          int32_t* ticket = a.tickets + worker_of(p.tile0, tiles, workers);
          last = atomicAdd(ticket, pages) + pages == p.np;
          if (last) *ticket = 0;
        }
      }
      s_last[tid] = last;
    }
    __syncthreads();
    for (int w = 0; w < W; ++w) {
      if (!s_last[w]) continue;
      __threadfence();
      join<HD, KEQV>(a, s_piece[w], tiles, workers, tid, C::kThreads);
    }
  }
  // ---- sequences without keys, and lengths that are wrong
  for (int b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
    const int len = __ldg(a.seq_lens + b);
    if (tid == 0 && (len < 0 || len > a.max_blocks * kBlockSize))
      flag_error(a.err, len < 0 ? PSW_DEVERR_LENGTH : PSW_DEVERR_CAPACITY);
    if (len > 0) continue;
    uint4* dst = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(b) * a.n_q * HD);
    for (int i = tid; i < a.n_q * (HD / 8); i += C::kThreads) dst[i] = make_uint4(0, 0, 0, 0);
    if (a.lse != nullptr)
      for (int i = tid; i < a.n_q; i += C::kThreads)
        a.lse[static_cast<int64_t>(b) * a.n_q + i] = -INFINITY;
  }
}

template <int HD, bool KEQV>
int launch(const Args& a, int num_sms, cudaStream_t stream) {
  using C = Cfg<HD, KEQV>;
  auto* fn = fp4_decode_kernel<HD, KEQV>;
  const int rc = set_smem_limit(reinterpret_cast<const void*>(fn), C::kSmem);
  if (rc != PSW_OK) return rc;
  const int grid = min(num_sms, kFp4MaxWorkers / C::kWarps);
  fn<<<grid, C::kThreads, C::kSmem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

int slot_rows(const LayerArgs& L) {
  const int heads = L.group() < kQHeadsPerUnit ? L.group() : kQHeadsPerUnit;
  return (heads + 1) / 2 * 2;
}

}  // namespace

size_t fp4_decode_workspace(const LayerArgs& L, int n_seqs) {
  const size_t slots = kFp4MaxWorkers + static_cast<size_t>(n_seqs) * L.n_kv * L.qchunks();
  return kFp4CounterBytes + slots * slot_rows(L) * (static_cast<size_t>(L.hd) * 4 + 8);
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
  a.num_blocks = pages.num_blocks;
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
  const size_t slots = kFp4MaxWorkers + static_cast<size_t>(n_seqs) * L.n_kv * L.qchunks();
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.tickets = reinterpret_cast<int32_t*>(w);
  a.ws_o = reinterpret_cast<float4*>(w + kFp4CounterBytes);
  a.ws_ml = reinterpret_cast<float2*>(w + kFp4CounterBytes + slots * a.rows * L.hd * 4);
  a.err = err;
  const StallHook hook = stall_hook(kStallDecode);
  a.stall_cta = hook.cta;
  a.stall_tile = hook.tile;
  if (L.hd == 256)
    return L.k_eq_v ? launch<256, true>(a, num_sms, stream) : launch<256, false>(a, num_sms, stream);
  return L.k_eq_v ? launch<512, true>(a, num_sms, stream) : launch<512, false>(a, num_sms, stream);
}

}  // namespace psw
