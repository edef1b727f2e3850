// fp4_cache.cu -- rows into 4-bit pages and back.
//
// Write: a head vector x of HD bf16 values becomes, per block of 16 values,
//   y = x * (1 / gs) in [-4096, 4096],  s = e4m3(max|y| / 6),  code = e2m1(y / s)
// (fp32 steps rounded to nearest; gs is the tensor's scale, given by the
// caller), so that code * s * gs stands for x. The division is the correctly
// rounded one: the codes' borders are numbers that y / s meets exactly, and a
// product with 1 / s would put some of those on the wrong side.
//
// A row has 2 HD bytes on one side and 9/16 HD on the other. On the GPU, inputs from memory: 8 chunks
// of 512 tokens, 4 KV heads, K and V (16.8 MB in) are written in 7.4 us, 2.2 of them start-up; 5
// ragged chunks of one tensor at HD 512 (25.7 MB in) in 8.7. What bounds the write behind its
// start is instructions: 134 for a row of 256 values, which take 7200 of the 11,600 cycles that an
// SM quarter is at work (9.4 us with 218: limits and products one at a time, rows of both tensors in a
// warp), 167 for a row of 512, 6900 of 14,400; memory is at 24 and 31 %. The read-back is bound by
// memory: 8 contexts of 512 to 8704 (391 MB in all) 68 us, 5.8 TB/s, four fifths of it stores.
#include "fp4.cuh"
#include "latent.cuh"

namespace psw {
namespace {

using fp4::Page;

constexpr int kWarps = 4;
constexpr uint32_t kMagnitudes = 0x7FFF7FFFu;
// Heads of a warp. Small blocks of little work, 16 of them on an SM (12 at HD 512): 64 tokens
// 2.2 us, 8 chunks of 512 7.4, ragged chunks 8.8; with 4 heads 2.4, 7.5 and 9.0, with 1 2.2, 9.3
// and 10.1.
constexpr int kRows = 2;

// Eight values (`v`) as codes: y / s of y = x * inv, given -s and 1 / s. LIMIT: where y may be
// an infinity or NaN, which the limits of y are for (finite magnitudes above 4096 become the
// largest code as 4096 does).
template <bool LIMIT>
__device__ __forceinline__ uint32_t codes_of(const uint4& v, float inv, float minus_s, float r) {
  const uint64_t inv2 = f2_pack(inv, inv), r2 = f2_pack(r, r), s2 = f2_pack(minus_s, minus_s);
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  float2 c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 xx = unpack_bf16x2(x[j]);
    uint64_t y = f2_mul(f2_pack(xx.x, xx.y), inv2);
    if (LIMIT) {
      const float2 z = f2_unpack(y);
      y = f2_pack(fmaxf(fminf(z.x, 4096.f), -4096.f), fmaxf(fminf(z.y, 4096.f), -4096.f));
    }
    c[j] = fp4::quotients(y, s2, r2);
  }
  return fp4::e2m1_codes(c);
}

// One warp takes kRows heads of one token and one tensor, the warps of a block neighbouring
// tokens: at HD 256 a lane holds 8 values of a head (a block is two lanes), at HD 512 16 (a block
// each). The rows are asked for before the token's sequence, page and slot are looked up.
template <int HD>
__global__ void __launch_bounds__(kWarps * 32, HD == 256 ? 16 : 12)
fp4_write_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                 const int32_t* __restrict__ cu_new, const int32_t* __restrict__ past_lens,
                 int n_seqs, int n_new_total, const int32_t* __restrict__ block_table,
                 int max_blocks, int64_t num_blocks, int n_kv, int groups, float k_inv,
                 float v_inv, uint8_t* __restrict__ k_pool, uint8_t* __restrict__ v_pool,
                 int32_t* err) {
  constexpr int kVec = HD / 256;  // 16-byte vectors per lane and row
  const int lane = threadIdx.x & 31;
  const uint32_t warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (warp >= static_cast<uint32_t>(n_new_total)) return;
  const int t = static_cast<int>(warp);
  const bool is_v = static_cast<int>(blockIdx.y) >= groups;
  const int head0 = (static_cast<int>(blockIdx.y) - (is_v ? groups : 0)) * kRows;
  const int total = __ldg(cu_new + n_seqs);
  const int heads = min(kRows, n_kv - head0);
  uint4 in[kRows][kVec];
  {
    const uint4* src = (is_v ? v : k) +
                       (static_cast<int64_t>(t) * n_kv + head0) * (HD / 8) + lane * kVec;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (i < heads) in[i][e] = __ldg(src + i * (HD / 8) + e);
  }
  // the token's sequence; up to 31 of them are looked at together with their past lengths
  int b = 0, start = 0, past = 0;
  bool found;
  if (n_seqs <= 31) {
    const int c = lane <= n_seqs ? __ldg(cu_new + lane) : 0;
    const int p = lane < n_seqs ? __ldg(past_lens + lane) : 0;
    const unsigned at = __ballot_sync(0xffffffffu, lane < n_seqs && c <= t);
    b = 31 - __clz(at);
    found = at != 0 && t < __shfl_sync(0xffffffffu, c, (b + 1) & 31);
    start = __shfl_sync(0xffffffffu, c, b & 31);
    past = __shfl_sync(0xffffffffu, p, b & 31);
  } else {
    found = lat::owner_of(cu_new, n_seqs, t, lane, b, start);
    if (found) past = __ldg(past_lens + b);
  }
  if (t == 0 && blockIdx.y == 0 && lane == 0 && total > n_new_total)
    flag_error(err, PSW_DEVERR_LENGTH);
  if (t >= total) return;
  if (!found) {
    if (lane == 0) flag_error(err, PSW_DEVERR_LENGTH);
    return;
  }
  const int64_t pos = static_cast<int64_t>(past) + (t - start);
  const int64_t page = pos / kBlockSize;
  if (past < 0 || page >= max_blocks) {  // (a negative past: no row of its sequence is written)
    if (lane == 0) flag_error(err, past < 0 ? PSW_DEVERR_LENGTH : PSW_DEVERR_CAPACITY);
    return;
  }
  const int32_t blk = __ldg(block_table + static_cast<int64_t>(b) * max_blocks + page);
  if (blk < 0 || blk >= num_blocks) {
    if (lane == 0) flag_error(err, PSW_DEVERR_BLOCK_ID);
    return;
  }
  const int r = static_cast<int>(pos % kBlockSize);
  const float inv = is_v ? v_inv : k_inv;
  uint8_t* to = (is_v ? v_pool : k_pool) +
                (static_cast<int64_t>(blk) * n_kv + head0) * Page<HD>::kBytes;
  uint8_t* codes = to + (HD == 256 ? Page<HD>::unit(r, lane >> 2) + (lane & 3) * 4
                                   : Page<HD>::unit(r, lane >> 1) + (lane & 1) * 8);
  uint8_t* scale = to + Page<HD>::scale(r, HD == 256 ? lane >> 1 : lane);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (i >= heads) break;
    // the largest |x| as bf16 bits; its product is the largest |y| (rounding keeps order)
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(in[i][e].x & kMagnitudes, in[i][e].y & kMagnitudes),
                                   __vmaxu2(in[i][e].z & kMagnitudes, in[i][e].w & kMagnitudes)));
    if (HD == 256) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const uint32_t big = max(top << 16, top & 0xFFFF0000u);
    const float peak = __fmul_rn(__uint_as_float(big), inv);
    const uint32_t s8 = fp4::block_scale(fminf(peak, 4096.f));  // (a NaN becomes the upper end)
    const float s = fp4::e4m3_float(s8);
    const float rs = fp4::scale_reciprocal(s);
    uint32_t w[kVec];
    if (__all_sync(0xffffffffu, peak < INFINITY)) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) w[e] = codes_of<false>(in[i][e], inv, -s, rs);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) w[e] = codes_of<true>(in[i][e], inv, -s, rs);
    }
    if constexpr (HD == 256) {
      *reinterpret_cast<uint32_t*>(codes + i * Page<HD>::kBytes) = w[0];
      if ((lane & 1) == 0) scale[i * Page<HD>::kBytes] = static_cast<uint8_t>(s8);
    } else {
      *reinterpret_cast<uint2*>(codes + i * Page<HD>::kBytes) = make_uint2(w[0], w[1]);
      scale[i * Page<HD>::kBytes] = static_cast<uint8_t>(s8);
    }
  }
}

}  // namespace

int launch_fp4_write(const LayerArgs& L, const void* k, const void* v, const int32_t* cu_new,
                     const int32_t* past_lens, int n_seqs, int n_new_total,
                     const psw_pages_t& pages, void* k_pool, void* v_pool, float k_scale,
                     float v_scale, int32_t* err, cudaStream_t stream) {
  const int groups = (L.n_kv + kRows - 1) / kRows, rows = groups * (L.k_eq_v ? 1 : 2);
  if (rows > 65535) return PSW_ECAPACITY;
  const dim3 grid((n_new_total - 1) / kWarps + 1, rows);
  auto* fn = L.hd == 256 ? fp4_write_kernel<256> : fp4_write_kernel<512>;
  fn<<<grid, kWarps * 32, 0, stream>>>(
      static_cast<const uint4*>(k), static_cast<const uint4*>(v), cu_new, past_lens, n_seqs,
      n_new_total, pages.block_table, pages.max_blocks_per_seq, pages.num_blocks, L.n_kv, groups,
      1.f / k_scale, 1.f / v_scale, static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool),
      err);
  return cudaGetLastError() == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

// ---------------------------------------------------------------- read-back
namespace {

// Four blocks on an SM; where each warp has many items, three of them do all: the memory
// takes the stores of fewer warps better (8 contexts of 512 to 8704: 67.6 us with 3, 70.5 with 4;
// 8 chunks of 512 8.1 and 7.7). With twice the threads and half the blocks 70.7 and 7.8.
constexpr int kReadThreads = 128;
constexpr int kReadBlocks = 4;
constexpr int kManyItems = 8;  // of a warp

// a / b: a division of 64 bits only where it takes one
__device__ __forceinline__ int64_t divided(int64_t a, uint32_t b) {
  return (a >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / b) : a / b;
}

// 32 bytes to a 16-byte aligned address; in one store where `wide` says that it is a
// multiple of 32 (two stores of 16 bytes each touch every sector twice: 8 contexts of 512 to
// 8704 tokens took 82.8 us with them, 73.4 without, in an earlier form).
__device__ __forceinline__ void store32(uint8_t* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// The pages wanted of all sequences form one list; with every (KV head, tensor) of a page, and
// every half (HD 256) or quarter (HD 512) of its tokens, they are the items, of which each
// warp of a persistent grid takes an equal run. A lane turns one block of 16 values (8 bytes and
// a scale) of a token into 32 bytes, so that a warp's store is whole rows: two tokens at HD 256,
// one at HD 512.
template <int HD>
__global__ void __launch_bounds__(kReadThreads, kReadBlocks)
fp4_read_kernel(const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool,
                const int32_t* __restrict__ table, int max_blocks, int64_t num_blocks,
                const int32_t* __restrict__ first, const int32_t* __restrict__ seq_lens,
                int n_seqs, const int32_t* __restrict__ out_table, int out_max_blocks,
                int64_t out_num_blocks, int n_kv, float k_scale, float v_scale,
                bool wide, uint8_t* __restrict__ k_out, uint8_t* __restrict__ v_out,
                int32_t* err) {
  constexpr int kTok = 512 / HD;               // tokens per warp store
  constexpr int kSteps = 4;                    // stores of an item
  constexpr int kSplit = kBlockSize / (kTok * kSteps);  // items of a page of a head
  constexpr int kLanes = HD / 16;              // lanes of a token
  __shared__ int s_run[kReadThreads + 1];
  __shared__ int s_warp[kReadThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = min(max_blocks, out_max_blocks) * kBlockSize;
  auto pages_of = [&](int b, bool flag) {
    int len = __ldg(seq_lens + b), lo = first != nullptr ? __ldg(first + b) : 0;
    if (len < 0 || lo < 0) {
      if (flag) flag_error(err, PSW_DEVERR_LENGTH);
      len = 0;
    } else if (len > cap) {
      if (flag) flag_error(err, PSW_DEVERR_CAPACITY);
      len = cap;
    }
    return fp4::seq_pages(len, max(lo, 0));
  };
  // pages before each thread's run of sequences
  const int per = (n_seqs + kReadThreads - 1) / kReadThreads;
  int mine = 0;
  for (int b = tid * per; b < min(n_seqs, (tid + 1) * per); ++b)
    mine += pages_of(b, blockIdx.x == 0).np;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < warp; ++i) before += s_warp[i];
  s_run[tid + 1] = before + incl;
  if (tid == 0) s_run[0] = 0;
  __syncthreads();
  const int rows = (v_out != nullptr ? 2 * n_kv : n_kv) * kSplit;  // items of a page
  const int64_t items = static_cast<int64_t>(s_run[kReadThreads]) * rows;
  int workers = gridDim.x * (kReadThreads / 32);
  if (items > static_cast<int64_t>(workers) * kManyItems) workers -= workers / kReadBlocks;
  const int me = blockIdx.x * (kReadThreads / 32) + warp;
  if (me >= workers) return;
  const int64_t each = divided(items, workers);
  const int more = static_cast<int>(items - each * workers);  // runs of an item more
  int64_t item = each * me + min(me, more);
  const int64_t end = item + each + (me < more ? 1 : 0);
  if (item >= end) return;
  // the sequence of the first item
  int page = static_cast<int>(divided(item, rows));
  int row = static_cast<int>(item - static_cast<int64_t>(page) * rows);
  int a = 0, z = kReadThreads;  // s_run[a] <= page < s_run[z]
  while (z - a > 1) {
    const int mid = (a + z) >> 1;
    if (s_run[mid] <= page) a = mid; else z = mid;
  }
  int b = a * per, off = s_run[a];
  fp4::SeqPages s = pages_of(b, false);
  while (page >= off + s.np) {
    off += s.np;
    s = pages_of(++b, false);
  }
  const int tok = lane / kLanes, blk16 = lane % kLanes;
  bool looked_up = false;
  int32_t src = 0, dst = 0;
  // what is on its way: an item's codes and scales, where its rows go, and which are wanted
  struct Asked {
    uint2 c[kSteps];
    uint32_t s8[kSteps];
    uint8_t* out;
    float gs;
    int lo, hi;
  };
  auto ask = [&](Asked& x) {
    if (!looked_up) {
      const int p = s.p0 + page - off;
      src = __ldg(table + static_cast<int64_t>(b) * max_blocks + p);
      dst = __ldg(out_table + static_cast<int64_t>(b) * out_max_blocks + p);
      if ((src < 0 || src >= num_blocks || dst < 0 || dst >= out_num_blocks) && row == 0 &&
          lane == 0)
        flag_error(err, PSW_DEVERR_BLOCK_ID);
      looked_up = true;
    }
    const int part = row / kSplit, r0 = (row - part * kSplit) * (kTok * kSteps) + tok;
    const bool is_v = part >= n_kv, have = src >= 0 && src < num_blocks;
    const int head = is_v ? part - n_kv : part, pos0 = (s.p0 + page - off) * kBlockSize + r0;
    const uint8_t* in = (is_v ? v_pool : k_pool) +
                        (static_cast<int64_t>(src) * n_kv + head) * Page<HD>::kBytes;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = r0 + i * kTok;
      x.c[i] = have ? __ldg(reinterpret_cast<const uint2*>(in + Page<HD>::unit(r, blk16 >> 1) +
                                                           (blk16 & 1) * 8))
                    : make_uint2(0, 0);
      x.s8[i] = have ? __ldg(in + Page<HD>::scale(r, blk16)) : 0;
    }
    x.out = (is_v ? v_out : k_out) +
            ((static_cast<int64_t>(dst) * kBlockSize + r0) * n_kv + head) * (HD * 2) + blk16 * 32;
    x.gs = is_v ? v_scale : k_scale;
    x.lo = s.lo - pos0;
    x.hi = dst >= 0 && dst < out_num_blocks ? s.len - pos0 : INT32_MIN;
    ++item;
    if (++row == rows) {
      row = 0;
      looked_up = false;
      ++page;
      while (item < end && page >= off + s.np) {
        off += s.np;
        s = pages_of(++b, false);
      }
    }
  };
  auto give = [&](const Asked& x) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const float f = fp4::e4m3_float(x.s8[i]) * x.gs;
      uint32_t w[8];
      const uint32_t cw[2] = {x.c[i].x, x.c[i].y};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t p[4] = {fp4::codes_f16<0>(cw[h]), fp4::codes_f16<1>(cw[h]),
                               fp4::codes_f16<2>(cw[h]), fp4::codes_f16<3>(cw[h])};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 y = fp4::f16x2_to_float2(p[j]);
          w[4 * h + j] = pack_bf16x2(y.x * f, y.y * f);
        }
      }
      if (i * kTok >= x.lo && i * kTok < x.hi)
        store32(x.out + static_cast<int64_t>(i * kTok) * n_kv * (HD * 2), w, wide);
    }
  };
  Asked now;
  ask(now);
  while (item < end) {  // (the next item is on its way while this one's rows are stored)
    Asked next;
    ask(next);
    give(now);
    now = next;
  }
  give(now);
}

}  // namespace

int launch_fp4_read(const LayerArgs& L, const void* k_pool, const void* v_pool,
                    const psw_pages_t& pages, const int32_t* first, const int32_t* seq_lens,
                    int n_seqs, const psw_pages_t& out_pages, void* k_out, void* v_out,
                    float k_scale, float v_scale, int num_sms, int32_t* err,
                    cudaStream_t stream) {
  const bool wide =
      ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) == 0;
  auto* fn = L.hd == 256 ? fp4_read_kernel<256> : fp4_read_kernel<512>;
  fn<<<num_sms * kReadBlocks, kReadThreads, 0, stream>>>(
      static_cast<const uint8_t*>(k_pool), static_cast<const uint8_t*>(v_pool), pages.block_table,
      pages.max_blocks_per_seq, pages.num_blocks, first, seq_lens, n_seqs, out_pages.block_table,
      out_pages.max_blocks_per_seq, out_pages.num_blocks, L.n_kv, k_scale, v_scale, wide,
      static_cast<uint8_t*>(k_out), static_cast<uint8_t*>(v_out), err);
  return cudaGetLastError() == cudaSuccess ? PSW_OK : PSW_ELAUNCH;
}

}  // namespace psw
