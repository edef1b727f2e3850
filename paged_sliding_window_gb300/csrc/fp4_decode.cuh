// fp4_decode.cuh -- the list of pages that the 4-bit decode works through, its cut into runs,
// the pieces that runs leave of units and their joining. Library-internal.
//
// Unit = (sequence, KV head, up to 8 query heads). The visible pages of all units form one list,
// in which every unit has some more entries (what it takes beside its pages); the workers of a
// persistent grid, one CTA per SM, have an equal run of it each.
//
// A worker's pieces: units that lie in its run alone are written out. Of the others it has at
// most two, the end of one unit (kept in the workspace, its CTA alone reads it) and the
// beginning or middle of another (left in shared memory where its ring of pages was). The CTA
// joins what its workers have of a unit; only units that other CTAs have pages of, two at most,
// go on to the workspace, and the warp that adds a unit's last pages (a ticket counts them)
// joins the CTAs' parts, in their order.
#pragma once

#include <type_traits>

#include "fp4.cuh"
#include "latent.cuh"

namespace psw {
namespace fp4 {

constexpr int kMaxCtas = 160;  // one per SM; what they need of workspace is counted with it
constexpr int kMaxWorkers = 12;  // of a CTA
constexpr int kMaxJobs = 8;    // parts of a unit's output that are joined apart, at most
constexpr int kGroup = 8;      // CTAs whose parts of a unit are joined first, where there are many
constexpr int kMostWhole = 1 << 16;  // pages of a unit that is not shared out among CTAs, at most
constexpr int kRuns = 256;     // runs of sequences whose entries are summed

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
  return i == 0 ? codes_f16<0>(w)
         : i == 1 ? codes_f16<1>(w)
         : i == 2 ? codes_f16<2>(w)
                  : codes_f16<3>(w);
}
__device__ __forceinline__ uint32_t word_at(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
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
  // [3][CTA][job]: pages joined of the unit that the CTA begins and does not end; of its first
  // group of CTAs; of the later group that begins with the CTA
  int32_t* tickets;
  int rows;          // rows of a slot: the group's heads, 8 at most, made even
  int32_t* err;
  int stall_cta, stall_tile;
};

struct Seq {
  int len, p0, np, lo;
};
__device__ __forceinline__ Seq seq_of_len(const Args& a, int len) {
  const int lo = a.window > 0 && len > a.window ? len - a.window : 0;
  const SeqPages s = seq_pages(len, lo);
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
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;"
               : "=r"(old) : "l"(p), "r"(v) : "memory");
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

// What a worker is given: the cut, its number, the unit that its run begins in with the
// first page there, and the entries of the run from that page on (none: nothing to do).
struct Run {
  Cut cut;
  int me, page, left;
  Place c;
};
struct ListSmem {
  int run[kRuns + 1], len[kRuns];  // len: where a run is one sequence
  int sum[kRuns / 32], most[kRuns / 32];
};

// W workers a CTA; called by all its threads (kRuns at least), with the worker that the calling
// warp is of. apart: what the joining of CTAs' parts takes, in pages of a CTA.
template <int W>
__device__ __forceinline__ Run begin_run(const Args& a, ListSmem& s, int worker, int cost,
                                         int apart) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ups = a.n_kv * a.qchunks;
  // entries of the sequences before each of kRuns runs of them
  const int per = (a.n_seqs + kRuns - 1) / kRuns;
  int incl = 0;
  if (tid < kRuns) {
    int most = 0;
    for (int b = tid * per; b < min(a.n_seqs, (tid + 1) * per); ++b) {
      const Seq q = seq_of(a, b);
      if (q.np > 0) incl += q.np + cost;
      most = max(most, q.np);
      s.len[tid] = q.len;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s.sum[warp] = incl;
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) s.most[warp] = most;
  }
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int i = 0; i < kRuns / 32; ++i) {
    if (i == warp) incl += all;
    all += s.sum[i];
  }
  if (tid < kRuns) s.run[tid + 1] = incl;
  if (tid == 0) s.run[0] = 0;
  __syncthreads();
  Run r;
  r.me = blockIdx.x * W + worker;
  r.page = r.left = 0;
  const int tiles = all * ups;
  // Where units are few and an equal share of all pages would save less than the joins take, a CTA
  // has whole units (one, or as many as divide its workers) and no part leaves it: 220
  // sequences of 1 or 2 with one KV head 8.0 us, cut into equal runs 10.9.
  {
    const int64_t ctas = gridDim.x, units = static_cast<int64_t>(a.n_seqs) * ups;
    int of_cta = 0, team = 0;
#pragma unroll
    for (int i = W; i >= 1; --i)
      if (W % i == 0 && units <= ctas * i) {
        of_cta = i;
        team = W / i;
      }
    int most = 0;
#pragma unroll
    for (int i = 0; i < kRuns / 32; ++i) most = max(most, s.most[i]);
    if (team > 0 && most <= kMostWhole && (most * of_cta - apart) * ctas <= tiles) {
      const int stretch = most + cost;  // (a worker's in the list, had it all these entries)
      const int mine = worker / team, unit = mine * gridDim.x + blockIdx.x;
      r.cut = Cut{stretch, 0};
      r.c.b = unit / ups;
      r.c.j = unit - r.c.b * ups;
      r.c.tile0 = (blockIdx.x * W + mine * team) * stretch;
      if (r.c.b < a.n_seqs) {
        r.c.s = per == 1 ? seq_of_len(a, s.len[r.c.b]) : seq_of(a, r.c.b);
        const int each = (r.c.s.np + team - 1) / team;
        r.page = (worker - mine * team) * each;
        r.left = max(0, min(each, r.c.s.np - r.page));
      }
      return r;
    }
  }
  // (two tiles each at least: a worker more is a piece more to join. One sequence of 40000 with
  // one KV head takes 17.4 us, with a tile each 18.9, with 3 or 4 one or two more)
  const int workers = max(1, min(static_cast<int>(gridDim.x) * W, tiles / 2));
  r.cut = Cut{tiles / workers, tiles % workers};
  if (r.me < min(workers, tiles)) {
    const int begin = r.cut.begin(r.me);
    r.left = r.cut.begin(r.me + 1) - begin;
    const int x = begin / ups;  // units of a sequence are equal: find its sequence by entries
    int lo = 31 - __clz(__ballot_sync(0xffffffffu, s.run[lane * (kRuns / 32)] <= x));
    lo = lo * (kRuns / 32);
    lo += 31 - __clz(__ballot_sync(0xffffffffu, lane < kRuns / 32 && s.run[lo + lane] <= x));
    Place c;
    c.b = lo * per;
    int off = s.run[lo];
    c.s = per == 1 ? seq_of_len(a, s.len[c.b]) : seq_of(a, c.b);
    while (c.s.np == 0 || x >= off + c.s.np + cost) {
      if (c.s.np > 0) off += c.s.np + cost;
      c.s = seq_of(a, ++c.b);
    }
    const int rem = begin - off * ups, entries = c.s.np + cost;
    c.j = rem / entries;
    const int at = rem - c.j * entries;
    c.tile0 = begin - at;
    r.page = max(0, at - cost);
    r.left -= max(0, cost - at);
    r.c = c;
  }
  return r;
}

// Joins the pieces of a CTA's W workers, WARPS warps, whose last pieces lie RING bytes apart in
// smem; weight: [2 W][8] floats of the calling warp's own.
template <int HD, int W, int WARPS, int RING>
__device__ __forceinline__ void join_pieces(const Args& a, const Cut& cut, int cost,
                                            const Piece (&s_piece)[2 * W],
                                            const float2 (&s_ml)[2 * W][kQHeadsPerUnit],
                                            const uint8_t* smem, float* weight) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ups = a.n_kv * a.qchunks, hp = a.rows / 2;
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
  const int units = (HD / 256) * 128 * hp;  // float4s of a unit
  const int64_t part0 = static_cast<int64_t>(gridDim.x) * W;  // slots of the CTAs' parts
  const int h = lane & 7, sub = lane >> 3;
  auto join = [&](auto per) {
    constexpr int PER = decltype(per)::value;
    const int jobs = units / (32 * PER);
    for (int y = warp; y < __popc(start) * jobs; y += WARPS) {
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
                          : __ldcg(a.ws_o +
                                   (static_cast<int64_t>(blockIdx.x) * W + (last >> 1)) * units +
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
          add(o[k], reinterpret_cast<const float4*>(smem + i * RING)[x0 + 32 * k],
              weight[(2 * i + 1) * 8 + head[k]]);
      }
      float top[PER], sum[PER];
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        top[k] = __shfl_sync(0xffffffffu, M, head[k]);
        sum[k] = __shfl_sync(0xffffffffu, L, head[k]);
      }
      if (pages != p.np) {  // other CTAs have pages of it: it is this CTA's first or last unit
        // Where many CTAs have, kGroup neighbours' parts are joined into one first (in the place
        // of the group's first), and the groups' then: one sequence of 40000 with one KV head
        // takes 17.4 us, with all its parts in a row 44.5.
        const Ctas cs = ctas_of<W>(cut, p, cost);
        const int64_t slot0 = part0 + cs.first + p.b * ups + p.j;  // of the first CTA's part
        const int at = static_cast<int>(blockIdx.x) - cs.first;
        // the parts from the `from`th on, n of them `step` apart: one pass with the running
        // maximum and sum of every lane's float4s
        auto add_parts = [&](int from, int step, int n) {
          const float4* src = a.ws_o + (slot0 + from) * units + x0;
          const float2* ml = a.ws_ml + ((slot0 + from) * jobs + job) * a.rows;
          const int so = step * units, sm = step * jobs * a.rows;
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            top[k] = -INFINITY;
            sum[k] = 0.f;
            o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll(8 / PER)
          for (int i = 0; i < n; ++i) {
            float4 v[PER];
            float2 x[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) {
              v[k] = __ldcg(src + static_cast<int64_t>(i) * so + 32 * k);
              x[k] = __ldcg(ml + static_cast<int64_t>(i) * sm + head[k]);
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
        };
        // adds what is ready to a ticket: whether that was the last of `want`
        auto last_of = [&](int32_t* ticket, int ready, int want) {
          __syncwarp();
          int done = 0;
          if (lane == 0) {
            done = add_acq_rel(ticket, ready) + ready == want;
            if (done) *ticket = 0;
          }
          done = __shfl_sync(0xffffffffu, done, 0);
          __syncwarp();
          return done != 0;
        };
        const int64_t slot = slot0 + at;
#pragma unroll
        for (int k = 0; k < PER; ++k) a.ws_o[slot * units + x0 + 32 * k] = o[k];
        if (lane < a.rows) a.ws_ml[(slot * jobs + job) * a.rows + lane] = make_float2(M, L);
        int32_t* ticket = a.tickets + cs.first * kMaxJobs + job;
        int ready = pages, step = 1, n = cs.n;
        if (n > 2 * kGroup) {
          const int from = at & ~(kGroup - 1), c0 = cs.first + from, m = min(kGroup, n - from);
          const int begin = p.tile0 + cost;
          ready = min(begin + p.np, cut.begin((c0 + m) * W)) - max(begin, cut.begin(c0 * W));
          int32_t* first = ticket + ((from == 0 ? 1 : 2) * kMaxCtas + from) * kMaxJobs;
          if (!last_of(first, pages, ready)) continue;
          add_parts(from, 1, m);
          __syncwarp();  // every lane has read the first part, whose place the group's takes
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            a.ws_o[(slot0 + from) * units + x0 + 32 * k] = o[k];
            a.ws_ml[((slot0 + from) * jobs + job) * a.rows + head[k]] = make_float2(top[k], sum[k]);
          }
          step = kGroup;
          n = (n + kGroup - 1) / kGroup;
        }
        if (!last_of(ticket, ready, p.np)) continue;
        add_parts(0, step, n);
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
}

// Zero rows for sequences without keys; lengths that are wrong are flagged.
template <int HD>
__device__ __forceinline__ void finish_empty(const Args& a) {
  const int tid = threadIdx.x;
  for (int b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
    const int len = __ldg(a.seq_lens + b);
    if (tid == 0 && (len < 0 || len > a.max_blocks * kBlockSize))
      flag_error(a.err, len < 0 ? PSW_DEVERR_LENGTH : PSW_DEVERR_CAPACITY);
    if (len > 0) continue;
    uint4* dst = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(b) * a.n_q * HD);
    for (int i = tid; i < a.n_q * (HD / 8); i += blockDim.x) dst[i] = make_uint4(0, 0, 0, 0);
    if (a.lse != nullptr)
      for (int i = tid; i < a.n_q; i += blockDim.x)
        a.lse[static_cast<int64_t>(b) * a.n_q + i] = -INFINITY;
  }
}

}  // namespace fp4
}  // namespace psw
