// fp4_decode.cu -- attention of one token per sequence over 4-bit pages.
//
//   s_j = scale * <q, K_j>, capped;  out = sum_j softmax(s)_j V_j
// over the keys that window and length leave, K_j and V_j being code * block
// scale * tensor scale. One kernel launch, bound by the pages' bytes where
// K and V are two pools, and by the conversion of codes next to that where one
// page serves as both (k_eq_v).
//
//  * Unit = (sequence, KV head, up to 8 query heads). The visible pages of all
//    units form one list, in which every unit has kUnitCost more entries; every warp of a persistent grid (one CTA per SM) is a
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
//  * A worker's pieces: units that lie in its run alone are written out. Of the
//    others it has at most two, the end of one unit (kept in the workspace, its CTA
//    alone reads it) and the beginning or middle of another (left in shared memory
//    where the ring was). The CTA joins what its warps have of a unit; only units
//    that other CTAs have pages of, two at most, go on to the workspace, and the warp
//    that adds a unit's last pages (a ticket counts them) joins the CTAs' parts, in
//    their order.
#include <type_traits>

#include "fp4.cuh"
#include "latent.cuh"

namespace psw {
namespace {

using fp4::Page;

constexpr int kMaxCtas = 160;  // one per SM; what they need of workspace is counted with it
constexpr int kMaxWarps = 12;
constexpr int kMaxJobs = 8;    // parts of a unit's output that are joined apart, at most
constexpr int kRuns = 256;     // runs of sequences whose entries are summed

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
  static constexpr int kQBytes = HD == 256 ? 0 : HD * 8 * 2;  // per warp: q as operands (HD 512)
  static constexpr int kSmem = kWarps * (kRingBytes + kQBytes);
  static_assert(kWarps <= kMaxWarps && 2 * kWarps <= 32, "pieces of a CTA");
  static_assert(kStages * kTileBytes == kRingBytes && kStages >= 2 && kStages <= 8, "ring");
  static_assert(HD * 8 * 4 <= kRingBytes, "a piece's output fits where the ring was");
  static_assert(HD * 8 * 4 + 2 * kWarps * 8 * 4 <= kRingBytes, "and its weights");
  static_assert(kMaxCtas * kMaxJobs * 4 <= PSW_FP4_COUNTER_BYTES && kMaxJobs == 8, "tickets");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
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
// The bounded wait of a whole warp: the same for all its lanes.
__device__ __forceinline__ bool landed(uint64_t* bar, uint32_t phase) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, phase));
}
// A bulk copy that only lanes with `p` ask for.
__device__ __forceinline__ void bulk_load_if(bool p, uint32_t dst, const void* src, uint32_t bytes,
                                             uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "@p cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
      "[%3];\n\t}" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "r"(static_cast<uint32_t>(p))
      : "memory");
}
__device__ __forceinline__ void expect_if(bool p, uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes), "r"(static_cast<uint32_t>(p))
      : "memory");
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
  int max_blocks, num_blocks;
  uint32_t page_stride;  // bytes of a block in a pool
  int n_seqs, n_q, n_kv, group, qchunks, window;
  float scale, softcap;  // scale: the layer's times K's tensor scale
  float v_scale;
  __nv_bfloat16* out;
  float* lse;
  float4* ws_o;      // [slot][half of a row's pairs ...], see piece_unit
  float2* ws_ml;     // [slot][job][rows]
  int32_t* tickets;  // [CTA][job]: pages joined of the unit that the CTA begins and does not end
  int rows;          // rows of a slot: the group's heads, 8 at most, made even
  int32_t* err;
  int stall_cta, stall_tile;
};

struct Seq {
  int len, p0, np, lo;
};
__device__ __forceinline__ Seq seq_of_len(const Args& a, int len) {
  const int lo = a.window > 0 && len > a.window ? len - a.window : 0;
  const fp4::SeqPages s = fp4::seq_pages(len, lo);
  return Seq{len, s.p0, s.np, lo};
}
__device__ __forceinline__ Seq seq_of(const Args& a, int b) {
  const int len = __ldg(a.seq_lens + b), cap = a.max_blocks * kBlockSize;
  return seq_of_len(a, len < 0 ? 0 : (len > cap ? cap : len));
}

// A unit of the list: sequence, unit of it, the list's index of its beginning.
struct Place {
  int b, j, tile0;
  Seq s;
  __device__ void next(const Args& a, int ups, int cost) {
    tile0 += s.np + cost;
    if (++j < ups) return;
    j = 0;
    do {
      s = seq_of(a, ++b);
    } while (s.np == 0);  // (only called where the list goes on)
  }
};

// The unit after a warp's `at`, which it becomes.
__device__ __forceinline__ Place next_place(Place* at, const Args& a, int ups, int cost) {
  Place p = *at;
  p.next(a, ups, cost);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) *at = p;
  __syncwarp();
  return p;
}

// Adds to a ticket: what this thread's warp has written before is seen by whoever sees the sum.
__device__ __forceinline__ int add_acq_rel(int32_t* p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// A unit's first query head, and how many it has.
__device__ __forceinline__ int first_head(const Args& a, int j) {
  return j / a.qchunks * a.group + j % a.qchunks * kQHeadsPerUnit;
}
__device__ __forceinline__ int heads_of(const Args& a, int j) {
  return min(kQHeadsPerUnit, a.group - j % a.qchunks * kQHeadsPerUnit);
}

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
  __nv_bfloat16* dst =
      a.out + (static_cast<int64_t>(p.b) * a.n_q + first_head(a, p.j) + u.head) * HD + u.d;
  const float f = inv * a.v_scale;
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
}
__device__ __forceinline__ void write_lse(const Args& a, const Piece& p, int head, float m,
                                          float l) {
  if (a.lse != nullptr)
    a.lse[static_cast<int64_t>(p.b) * a.n_q + first_head(a, p.j) + head] =
        (m + log2f(l)) * lat::kLn2;
}


// The list of `tiles` entries cut into runs for `workers`: of each + 1 entries for the first
// `more` of them, of `each` for the others.
struct Cut {
  int each, more;
  __device__ int begin(int w) const { return w * each + min(w, more); }
  __device__ int worker(int x) const {  // that has entry x
    const int y = x - more * (each + 1);
    return y < 0 ? x / (each + 1) : more + y / each;
  }
};

// The CTAs (of W workers) that have pages of a unit: the first of them and how many.
struct Ctas {
  int first, n;
};
template <int W>
__device__ __forceinline__ Ctas ctas_of(const Cut& cut, const Piece& p, int cost) {
  const int first = cut.worker(p.tile0 + cost) / W;
  return Ctas{first, cut.worker(p.tile0 + cost + p.np - 1) / W - first + 1};
}

template <int HD, bool KEQV>
__global__ void __launch_bounds__(Cfg<HD, KEQV>::kThreads, 1) fp4_decode_kernel(const Args a) {
  using C = Cfg<HD, KEQV>;
  constexpr int W = C::kWarps, S = C::kStages, TP = C::kTile;
  constexpr int kUnitCost = fp4_unit_cost(HD);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_full[W][S];
  __shared__ Piece s_piece[2 * W];
  __shared__ float2 s_ml[2 * W][kQHeadsPerUnit];
  __shared__ int s_run[kRuns + 1], s_len[kRuns];  // s_len: where a run is one sequence
  __shared__ int s_sum[kRuns / 32];
  // a warp's unit that is worked on, and that of the next page to fetch: wanted at a unit's
  // ends alone, and no registers are to spare between them
  __shared__ Place s_now[W], s_next[W];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::kRingBytes;
  const int ups = a.n_kv * a.qchunks, hp = a.rows / 2;

  // ---- the list: entries of the sequences before each run of them
  if (lane < S) mbar_init(&s_full[warp][lane], 1);
  fence_mbar_init();
  const int per = (a.n_seqs + kRuns - 1) / kRuns;
  int incl = 0;
  if (tid < kRuns) {
    for (int b = tid * per; b < min(a.n_seqs, (tid + 1) * per); ++b) {
      const Seq s = seq_of(a, b);
      if (s.np > 0) incl += s.np + kUnitCost;
      s_len[tid] = s.len;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_sum[warp] = incl;
  }
  if (tid < 2 * W) s_piece[tid].pages = 0;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int i = 0; i < kRuns / 32; ++i) {
    if (i == warp) incl += all;
    all += s_sum[i];
  }
  if (tid < kRuns) s_run[tid + 1] = incl;
  if (tid == 0) s_run[0] = 0;
  __syncthreads();
  const int tiles = all * ups;
  const int workers = max(1, min(static_cast<int>(gridDim.x) * W, tiles));
  const Cut cut{tiles / workers, tiles % workers};
  const int me = blockIdx.x * W + warp;

  int page = 0;   // the next page of the unit that is worked on
  int np = 0;     // its pages
  int left = 0;   // entries of the run from the next page to fetch on
  if (me < min(workers, tiles)) {
    const int begin = cut.begin(me);
    left = cut.begin(me + 1) - begin;
    const int x = begin / ups;  // units of a sequence are equal: find its sequence by entries
    int lo = 31 - __clz(__ballot_sync(0xffffffffu, s_run[lane * (kRuns / 32)] <= x));
    lo = lo * (kRuns / 32);
    lo += 31 - __clz(__ballot_sync(0xffffffffu, lane < kRuns / 32 && s_run[lo + lane] <= x));
    Place c;
    c.b = lo * per;
    int off = s_run[lo];
    c.s = per == 1 ? seq_of_len(a, s_len[c.b]) : seq_of(a, c.b);
    while (c.s.np == 0 || x >= off + c.s.np + kUnitCost) {
      if (c.s.np > 0) off += c.s.np + kUnitCost;
      c.s = seq_of(a, ++c.b);
    }
    const int rem = begin - off * ups, entries = c.s.np + kUnitCost;
    c.j = rem / entries;
    const int at = rem - c.j * entries;
    c.tile0 = begin - at;
    page = max(0, at - kUnitCost);
    left -= max(0, kUnitCost - at);
    np = c.s.np;
    if (lane == 0) s_now[warp] = s_next[warp] = c;
    __syncwarp();
  }
  if (left > 0) {
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
    float acc[HD / 16][4];    // value 32 g + 2 i (+ 256 part): heads 2 t, 2 t + 1; the next value: same
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
      const float fac = a.scale * down * (a.softcap > 0.f ? 1.f / a.softcap : lat::kLog2e);
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
      float s[TP][4];
#pragma unroll
      for (int pg = 0; pg < TP; ++pg)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[pg][x] = 0.f;
      {
        uint32_t ks[TP][2][HD / 256];  // scale bytes of tokens r0, r0 + 8: two blocks per 128 values
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
            const uint8_t* p = tile + pg * C::kPageBytes + (k >> 1) * 2048 + (k_at ^ ((k & 1) * 64));
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
                const uint32_t wa = jp == 0 ? ka[pg].x : jp == 1 ? ka[pg].y : jp == 2 ? ka[pg].z : ka[pg].w;
                const uint32_t wb = jp == 0 ? kb[pg].x : jp == 1 ? kb[pg].y : jp == 2 ? kb[pg].z : kb[pg].w;
                const uint32_t x[4] = {mul_f16x2(codes_at(wa, 2 * half), ea[pg][h]),
                                       mul_f16x2(codes_at(wb, 2 * half), eb[pg][h]),
                                       mul_f16x2(codes_at(wa, 2 * half + 1), ea[pg][h]),
                                       mul_f16x2(codes_at(wb, 2 * half + 1), eb[pg][h])};
                mma_f16(s[pg], x, half ? qq.z : qq.x, half ? qq.w : qq.y);
              }
          }
        }
      }
      // ---- softmax: tokens r0, r0 + 8 of heads 2 t, 2 t + 1
      float z[TP][4];
#pragma unroll
      for (int pg = 0; pg < TP; ++pg)
#pragma unroll
        for (int x = 0; x < 4; ++x) z[pg][x] = s[pg][x] * qf[x & 1];
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

  // ---- joining: the pieces of a unit are neighbours. A warp takes a part of what the CTA has of a
  // unit at a time (32 PER float4) and needs no other warp for the rest of the way: it writes
  // the result, or this CTA's part and, if its part is the last to come, the result of all.
  const Piece mine = s_piece[min(lane, 2 * W - 1)];
  const bool valid = lane < 2 * W && mine.pages > 0;
  const uint32_t have = __ballot_sync(0xffffffffu, valid);
  uint32_t start;  // the first piece of every unit
  {
    const uint32_t prev = have & ((1u << lane) - 1u);
    const int other = __shfl_sync(0xffffffffu, mine.tile0, prev != 0 ? 31 - __clz(prev) : 0);
    start = __ballot_sync(0xffffffffu, valid && (prev == 0 || other != mine.tile0));
  }
  const int units = C::kParts * 128 * hp;  // float4s of a unit
  const int64_t part0 = static_cast<int64_t>(gridDim.x) * W;  // slots of the CTAs' parts
  float* weight = reinterpret_cast<float*>(ring + HD * 8 * 4);  // [piece][head], of this warp
  const int h = lane & 7, sub = lane >> 3;
  auto join = [&](auto per) {
    constexpr int PER = decltype(per)::value;
    const int jobs = units / (32 * PER);
    for (int y = warp; y < __popc(start) * jobs; y += W) {
      const int gi = y / jobs, job = y - gi * jobs, x0 = job * 32 * PER + lane;
      uint32_t from = start;
      for (int k = 0; k < gi; ++k) from &= from - 1;
      const int first = __ffs(from) - 1;
      from &= from - 1;  // the starts behind it
      const uint32_t members =
          have & ~((1u << first) - 1u) & (from != 0 ? (from & -from) - 1u : ~0u);
      // (a first piece can only be the last of a unit: the run that it begins goes on elsewhere)
      const int last = 31 - __clz(members);
      float4 o[PER];
      int head[PER];
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        head[k] = piece_unit(x0 + 32 * k, hp).head;
        o[k] = (last & 1) ? make_float4(0.f, 0.f, 0.f, 0.f)
                          : __ldcg(a.ws_o + (static_cast<int64_t>(blockIdx.x) * W + (last >> 1)) * units +
                                   x0 + 32 * k);
      }
      const int pages = __reduce_add_sync(0xffffffffu, (members >> lane) & 1 ? mine.pages : 0);
      Piece p;
      p.b = __shfl_sync(0xffffffffu, mine.b, first);
      p.j = __shfl_sync(0xffffffffu, mine.j, first);
      p.tile0 = __shfl_sync(0xffffffffu, mine.tile0, first);
      p.np = __shfl_sync(0xffffffffu, mine.np, first);
      const int nh = heads_of(a, p.j);
      const int w0 = first >> 1, w1 = (last - 1) >> 1;  // its last pieces
      // M = max m_i, weights 2^(m_i - M), their sum of l; a lane has every fourth piece of head h
      float M = -INFINITY, L = 0.f;
      for (int i = first + sub; i <= last; i += 4)
        if ((members >> i) & 1) M = fmaxf(M, s_ml[i][h].x);
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
      __syncwarp();
      for (int i = first + sub; i <= last; i += 4) {
        if (!((members >> i) & 1)) continue;
        const float2 ml = s_ml[i][h];
        const float w = ex2_approx(ml.x - M);
        weight[i * 8 + h] = w;
        L += w * ml.y;
      }
      L += __shfl_xor_sync(0xffffffffu, L, 8);
      L += __shfl_xor_sync(0xffffffffu, L, 16);
      __syncwarp();
      auto add = [](float4& s, const float4& v, float w) {
        s.x += v.x * w;
        s.y += v.y * w;
        s.z += v.z * w;
        s.w += v.w * w;
      };
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const float w = (last & 1) ? 0.f : weight[last * 8 + head[k]];
        o[k] = make_float4(o[k].x * w, o[k].y * w, o[k].z * w, o[k].w * w);
      }
#pragma unroll 2
      for (int i = w0; i <= w1; ++i) {
#pragma unroll
        for (int k = 0; k < PER; ++k)
          add(o[k], reinterpret_cast<const float4*>(smem + i * C::kRingBytes)[x0 + 32 * k],
              weight[(2 * i + 1) * 8 + head[k]]);
      }
      float top[PER], sum[PER];
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        top[k] = __shfl_sync(0xffffffffu, M, head[k]);
        sum[k] = __shfl_sync(0xffffffffu, L, head[k]);
      }
      if (pages != p.np) {  // other CTAs have pages of it: it is this CTA's first or last unit
        const Ctas cs = ctas_of<W>(cut, p, kUnitCost);
        const int64_t slot0 = part0 + cs.first + p.b * ups + p.j;  // of the first CTA's part
        const int64_t slot = slot0 + static_cast<int>(blockIdx.x) - cs.first;
#pragma unroll
        for (int k = 0; k < PER; ++k) a.ws_o[slot * units + x0 + 32 * k] = o[k];
        if (lane < a.rows) a.ws_ml[(slot * jobs + job) * a.rows + lane] = make_float2(M, L);
        __syncwarp();
        int done = 0;
        if (lane == 0) {
          int32_t* ticket = a.tickets + cs.first * kMaxJobs + job;
          done = add_acq_rel(ticket, pages) + pages == p.np;
          if (done) *ticket = 0;
        }
        if (__shfl_sync(0xffffffffu, done, 0) == 0) continue;
        __syncwarp();
        // one pass over the parts with the running maximum and sum of every lane's float4s
        const float4* src = a.ws_o + slot0 * units + x0;
        const float2* ml = a.ws_ml + (slot0 * jobs + job) * a.rows;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          top[k] = -INFINITY;
          sum[k] = 0.f;
          o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll(8 / PER)
        for (int i = 0; i < cs.n; ++i) {
          float4 v[PER];
          float2 x[PER];
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            v[k] = __ldcg(src + static_cast<int64_t>(i) * units + 32 * k);
            x[k] = __ldcg(ml + static_cast<int64_t>(i) * jobs * a.rows + head[k]);
          }
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            const float mn = fmaxf(top[k], x[k].x);
            const float f0 = top[k] == mn ? 1.f : ex2_approx(top[k] - mn);
            const float f1 = ex2_approx(x[k].x - mn);
            top[k] = mn;
            sum[k] = sum[k] * f0 + x[k].y * f1;
            o[k] = make_float4(o[k].x * f0, o[k].y * f0, o[k].z * f0, o[k].w * f0);
            add(o[k], v[k], f1);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const Unit4 u = piece_unit(x0 + 32 * k, hp);
        write_out<HD>(a, p, nh, u, o[k], 1.f / sum[k]);
        if (u.d == 0 && u.head < nh) write_lse(a, p, u.head, top[k], sum[k]);
      }
    }
  };
  // (2: more warps share few heads' units; 4: fewer rounds where there are many, and kMaxJobs
  // parts at most. 64 sequences of 64 pages, G 2: 35.8 us with 2, 38.2 with 1, 36.2 with 4)
  if (units <= 256) {
    join(std::integral_constant<int, 2>{});
  } else {
    join(std::integral_constant<int, 4>{});
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
  return kMaxCtas * (kMaxWarps + 1) + static_cast<size_t>(n_seqs) * L.n_kv * L.qchunks();
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
    return L.k_eq_v ? launch<256, true>(a, num_sms, stream) : launch<256, false>(a, num_sms, stream);
  return L.k_eq_v ? launch<512, true>(a, num_sms, stream) : launch<512, false>(a, num_sms, stream);
}

}  // namespace psw
