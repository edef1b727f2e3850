// block_tables.cu -- the tables of a step from its requests' lengths: offsets,
// lengths, new block-table entries and the slots of the new tokens.
//
// With need(b) = pages(past + new) - pages(past) and the sequences in order, the
// k-th page needed of all is free_ids[free_pos + k]. Everything follows from two
// prefix sums (tokens and pages), so the work is two scans and then one thread
// for each new page and each new token; it is bound by latency: the lengths are
// read, scanned, looked up and written (64 decoding sequences 3.7 us on the GPU, 256
// and four chunks of 2048 tokens 5.3).
#include "psw_internal.h"
#include "ptx.cuh"

namespace psw {
namespace {

constexpr int kThreads = 1024;
constexpr int kWideCtas = 8;  // a cluster of these where there are many tokens

// Pages of n tokens (n up to INT32_MAX).
__device__ __forceinline__ int pages_of(int n) {
  return n / kBlockSize + (n % kBlockSize != 0);
}

// Exclusive prefix sum over the block; *total is the sum.
template <class T>
__device__ __forceinline__ T block_scan(T x, T* s_warp, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    T w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  const T before = warp > 0 ? s_warp[warp - 1] : T(0);
  __syncthreads();  // s_warp may be used again
  return before + incl - x;
}

// The last i below n with s[i] <= x (s[0] <= x).
template <class T>
__device__ __forceinline__ int last_at_most(const T* s, int n, T x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// One cluster (of one CTA or of kWideCtas). Sequences are taken kThreads at a
// time, one a thread; every CTA scans them all, and the pages and tokens that
// they bring are shared out among all threads of the cluster. Without sequences (free_next is
// then not free_pos) the offsets' end and the cursor are all there is to write.
__global__ void __launch_bounds__(kThreads)
block_table_extend_kernel(int32_t* block_table, int max_blocks, const int32_t* past_lens,
                          const int32_t* new_lens, int n_seqs, const int32_t* free_ids,
                          int n_free, const int32_t* free_pos, int32_t* free_next,
                          int32_t* cu_new, int32_t* seq_lens, int64_t* slots, int n_slots,
                          int32_t* err) {
  __shared__ int64_t s_tok[kThreads + 1];
  __shared__ int32_t s_page[kThreads + 1];
  __shared__ int32_t s_past[kThreads];
  __shared__ int64_t s_warp64[32];
  __shared__ int32_t s_warp32[32];
  const int tid = threadIdx.x;
  const int rank = blockIdx.x, ctas = gridDim.x;
  const int all = ctas * kThreads, me = rank * kThreads + tid;
  int pos0 = *free_pos;
  const bool bad_pos = pos0 < 0 || pos0 > n_free;
  // every CTA has read the cursor before the first one writes the next
  if (ctas > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (bad_pos) pos0 = n_free;
  const int avail = n_free - pos0;
  int32_t bits = bad_pos ? PSW_DEVERR_LENGTH : 0;
  int64_t tok0 = 0;
  int page0 = 0;
  for (int base = 0; base < n_seqs; base += kThreads) {
    const int b = base + tid, n = min(kThreads, n_seqs - base);
    int past = 0, add = 0, need = 0;
    if (tid < n) {
      past = past_lens[b];
      add = new_lens[b];
      if (past < 0 || add < 0 || static_cast<int64_t>(past) + add > INT32_MAX - kBlockSize) {
        bits |= PSW_DEVERR_LENGTH;
        past = max(past, 0);
        add = 0;
      }
      const int have = pages_of(past), want = pages_of(past + add);
      if (want > max_blocks) bits |= PSW_DEVERR_CAPACITY;
      need = max(0, min(want, max_blocks) - have);
    }
    int64_t toks;
    int pages;
    const int64_t t_before = block_scan<int64_t>(add, s_warp64, &toks);
    const int p_before = block_scan<int32_t>(need, s_warp32, &pages);
    s_tok[tid] = t_before;
    s_page[tid] = p_before;
    s_past[tid] = past;
    if (rank == 0 && tid < n) {
      cu_new[b] = static_cast<int32_t>(min(tok0 + t_before, static_cast<int64_t>(INT32_MAX)));
      seq_lens[b] = past + add;
    }
    __syncthreads();
    for (int k = me; k < pages; k += all) {
      const int i = last_at_most(s_page, n, k);
      const int have = pages_of(s_past[i]);
      const int at = page0 + k;
      int32_t id = -1;
      if (at < avail) id = free_ids[pos0 + at]; else bits |= PSW_DEVERR_NOBLOCKS;
      block_table[static_cast<int64_t>(base + i) * max_blocks + have + (k - s_page[i])] = id;
    }
    if (slots != nullptr) {
      const int64_t room = n_slots - tok0;
      if (toks > room) bits |= PSW_DEVERR_LENGTH;
      for (int64_t t = me; t < min(toks, room); t += all) {
        const int i = last_at_most(s_tok, n, t);
        const int pos = s_past[i] + static_cast<int>(t - s_tok[i]);
        const int have = pages_of(s_past[i]), page = pos / kBlockSize;
        int32_t id = -1;
        if (page < max_blocks) {
          if (page < have) {
            id = block_table[static_cast<int64_t>(base + i) * max_blocks + page];
            if (id < 0) bits |= PSW_DEVERR_BLOCK_ID;
          } else {
            const int at = page0 + s_page[i] + (page - have);
            if (at < avail) id = free_ids[pos0 + at];
          }
        }
        slots[tok0 + t] = id < 0 ? -1 : static_cast<int64_t>(id) * kBlockSize + pos % kBlockSize;
      }
    }
    tok0 += toks;
    page0 += pages;
    __syncthreads();  // the next sequences take the arrays
  }
  if (tok0 > INT32_MAX) bits |= PSW_DEVERR_LENGTH;
  if (bits != 0) flag_error(err, bits);
  if (ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && tid == 0) {
    cu_new[n_seqs] = static_cast<int32_t>(min(tok0, static_cast<int64_t>(INT32_MAX)));
    *free_next = pos0 + min(page0, avail);
  }
}

}  // namespace

int launch_block_table_extend(int32_t* block_table, int max_blocks, const int32_t* past_lens,
                              const int32_t* new_lens, int n_seqs, const int32_t* free_ids,
                              int n_free, const int32_t* free_pos, int32_t* free_next,
                              int32_t* cu_new, int32_t* seq_lens, int64_t* slots, int n_slots,
                              int32_t* err, cudaStream_t stream) {
  const int ctas = n_slots > 2 * kThreads ? kWideCtas : 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_table_extend_kernel, block_table, max_blocks, past_lens,
                            new_lens, n_seqs, free_ids, n_free, free_pos, free_next, cu_new,
                            seq_lens, slots, n_slots, err) == cudaSuccess
             ? PSW_OK
             : PSW_ELAUNCH;
}

}  // namespace psw
