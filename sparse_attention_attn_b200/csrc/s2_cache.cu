// Blocks, slots, positions and ancestor masks of the new tokens of a batch
// that extends a paged cache, built on the GPU from the requests' lengths.
//
// Request i holds ctx_i tokens in ceil(ctx_i / bs) blocks and gains new_i; the
// blocks it then lacks come off the free list in request order.  Token j of
// request i lies at place p = ctx_i + j: block block_table[i][p / bs], row
// p % bs.  In a tree of drafts (parents given) its position is ctx_i plus its
// depth, and its mask has bit j' for itself and each of its ancestors.
//
// The work is a few bytes a token, so launch and latency bound it: one launch,
// each block of 256 threads takes 256 tokens and scans the requests' lengths
// itself (they sit in L2) up to its window instead of waiting for a scan
// kernel.  A request that overlaps the window leaves a marker at its first
// token there; a maximum scan of the markers gives every token its request.
// No block reads what another writes: the entries of new blocks are computed
// from the free list, and only entries that were there before are read.
#include <cuda.h>
#include <cuda_runtime.h>

#include "s2_common.cuh"

namespace s2 {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanPer = 4;       // requests a thread scans at a time
constexpr int kPlanBack = 63;     // drafts before the window whose parents are staged (a mask has 64 bits)

__global__ void __launch_bounds__(kPlanThreads) s2_cache_plan_kernel(CachePlanArgs a) {
  __shared__ int marker[kPlanThreads], req[kPlanThreads], cu[kPlanThreads], first[kPlanThreads];
  __shared__ int par[kPlanBack + kPlanThreads];
  __shared__ unsigned long long wsum[kPlanThreads / 32];
  __shared__ int wmax[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long t0 = static_cast<long long>(blockIdx.x) * kPlanThreads, t1 = t0 + kPlanThreads;
  const uint32_t bs = a.block_size;
  marker[tid] = -1;
  if (a.parents != nullptr)
    for (int x = tid; x < kPlanBack + kPlanThreads; x += kPlanThreads) {
      const long long t = t0 - kPlanBack + x;
      par[x] = t >= 0 && t < a.T ? a.parents[t] : -1;
    }
  __syncthreads();
  unsigned long long run = 0;  // tokens (high word) and new blocks (low word) before this chunk
  unsigned long long lost = 0;
  for (int base = 0; base < a.R; base += kPlanThreads * kPlanPer) {
    unsigned long long v[kPlanPer], sum = 0;
    int ctx[kPlanPer], n[kPlanPer];
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      const int i = base + tid * kPlanPer + k;
      ctx[k] = i < a.R ? max(a.ctx_lens[i], 0) : 0;
      n[k] = i < a.R ? max(a.new_lens[i], 0) : 0;
      const uint32_t have = min((static_cast<uint32_t>(ctx[k]) + bs - 1) / bs, static_cast<uint32_t>(a.max_blocks));
      const uint32_t need = min(static_cast<uint32_t>((static_cast<unsigned long long>(ctx[k]) + n[k] + bs - 1) / bs),
                                static_cast<uint32_t>(a.max_blocks));
      v[k] = static_cast<unsigned long long>(n[k]) << 32 | (need - have);
      sum += v[k];
    }
    unsigned long long inc = sum;  // inclusive scan over the block
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const unsigned long long o = __shfl_up_sync(0xffffffffu, inc, m);
      if (lane >= m) inc += o;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    unsigned long long before = run, all = run;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) before += wsum[w];
      all += wsum[w];
    }
    unsigned long long at = before + inc - sum;
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      const int i = base + tid * kPlanPer + k;
      const long long c = static_cast<long long>(at >> 32);
      const uint32_t f = static_cast<uint32_t>(at);
      if (i < a.R) {
        if (blockIdx.x == 0) {
          a.cu_seqlens[i] = static_cast<int>(c);
          // places below `end` have a block: the table's width, and what is left of the free list
          const uint32_t have = min((static_cast<uint32_t>(ctx[k]) + bs - 1) / bs, static_cast<uint32_t>(a.max_blocks));
          const uint32_t left = f < static_cast<uint32_t>(a.num_free) ? a.num_free - f : 0u;
          const uint32_t got = min(static_cast<uint32_t>(v[k]), left);
          const long long last = static_cast<long long>(ctx[k]) + n[k];
          const long long end = max(static_cast<long long>(have + got) * bs, static_cast<long long>(ctx[k]));
          if (last > end) lost += last - end;
        }
        if (n[k] > 0 && c < t1 && c + n[k] > t0) {
          const int p = static_cast<int>((c > t0 ? c : t0) - t0);
          marker[p] = p;
          req[p] = i;
          cu[p] = static_cast<int>(c);
          first[p] = static_cast<int>(f);
        }
      }
      at += v[k];
    }
    run = all;
    __syncthreads();  // wsum is reused; markers are complete after the last chunk
    if (blockIdx.x != 0 && static_cast<long long>(run >> 32) > t1) break;  // (the last block sees whether tokens are dropped)
  }
  if (blockIdx.x == 0) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) lost += __shfl_xor_sync(0xffffffffu, lost, m);
    if (lane == 0) wsum[warp] = lost;
    __syncthreads();
    if (tid == 0) {
      unsigned long long l = 0;
      for (int w = 0; w < kPlanThreads / 32; ++w) l += wsum[w];
      const uint32_t needed = static_cast<uint32_t>(run);
      a.cu_seqlens[a.R] = static_cast<int>(run >> 32);
      if (static_cast<long long>(run >> 32) <= a.T)  // (else the last token kept writes it)
        a.counts[0] = static_cast<int>(min(needed, static_cast<uint32_t>(a.num_free)));
      a.counts[1] = static_cast<int>(needed);
      a.counts[2] = static_cast<int>(run >> 32);
      a.counts[3] = static_cast<int>(l);
    }
  }
  // the request of every token of the window: the last marker at or before it
  int m = marker[tid];
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, m, s);
    if (lane >= s) m = max(m, o);
  }
  if (lane == 31) wmax[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w)
    if (w < warp) m = max(m, wmax[w]);
  const long long t = t0 + tid;
  if (t >= a.T) return;
  if (m < 0 || t >= static_cast<long long>(run >> 32)) {  // padding behind the last request
    a.positions[t] = 0;
    a.slots[t] = -1;
    if (a.mask != nullptr) a.mask[t] = 0ull;
    return;
  }
  const int i = req[m], j = static_cast<int>(t) - cu[m], ctx = max(a.ctx_lens[i], 0);
  const uint32_t place = static_cast<uint32_t>(ctx) + static_cast<uint32_t>(j);
  const uint32_t col = place / bs, row = place - col * bs;
  const uint32_t have = min((static_cast<uint32_t>(ctx) + bs - 1) / bs, static_cast<uint32_t>(a.max_blocks));
  // the last token kept, others behind it dropped: the blocks up to its own are taken
  if (t == a.T - 1 && static_cast<long long>(run >> 32) > a.T) {
    const uint32_t opened = first[m] + max(min(col + 1, static_cast<uint32_t>(a.max_blocks)), have) - have;
    a.counts[0] = static_cast<int>(min(opened, static_cast<uint32_t>(a.num_free)));
  }
  int blk = -1;
  if (col < static_cast<uint32_t>(a.max_blocks)) {
    int* entry = a.block_tables + static_cast<size_t>(i) * a.max_blocks + col;
    if (!in_bounds(a.status, i, a.R, 730)) {
      blk = -1;
    } else if (col < have) {
      blk = *entry;
    } else {
      const uint32_t f = static_cast<uint32_t>(first[m]) + (col - have);
      if (f < static_cast<uint32_t>(a.num_free)) blk = a.free_blocks[f];
      if (row == 0) *entry = blk;  // the block's first token writes the table
    }
  }
  const long long slot = static_cast<long long>(blk) * bs + row;
  a.slots[t] = blk < 0 || slot > 0x7fffffffLL ? -1 : static_cast<int>(slot);
  int depth = j;
  if (a.parents != nullptr) {
    unsigned long long bits = j < 64 ? 1ull << j : 0ull;
    depth = 0;
    int at = j;
    for (;;) {
      const long long x = static_cast<long long>(cu[m]) + at - (t0 - kPlanBack);
      if (!in_bounds(a.status, x >= 0 ? x : 0, kPlanBack + kPlanThreads, 731) ||
          !in_bounds(a.status, static_cast<long long>(cu[m]) + at, a.T, 732))
        break;
      const int up = x >= 0 ? par[x] : a.parents[static_cast<long long>(cu[m]) + at];
      if (up < 0 || up >= at) break;  // a parent comes before its child
      if (up < 64) bits |= 1ull << up;
      ++depth;
      at = up;
    }
    a.mask[t] = bits;
  }
  a.positions[t] = ctx + depth;
}

}  // namespace

cudaError_t launch_cache_plan(const CachePlanArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const int grid = static_cast<int>((static_cast<long long>(a.T) + kPlanThreads - 1) / kPlanThreads);
  prof_before(stream, kKernelCachePlan);
  s2_cache_plan_kernel<<<grid, kPlanThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  prof_after(stream);
  return e;
}

}  // namespace s2
