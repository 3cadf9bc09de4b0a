// What the two cache attention kernels (s2_cache_dec.cu, s2_cache_tc.cu) share:
// the numbering of the work and its split over the CTAs, and the join of items
// that more than one CTA worked on.
//
// An item is the new tokens of one row tile (or pair of tiles) of one (request,
// kv head) against all of the request's keys; a unit is one key tile of an
// item.  All units of a batch are numbered request by request and dealt to the
// CTAs in equal contiguous runs, so that a batch of very different lengths, or
// one long request, loads every SM alike.  A segment is the part of an item
// that lies in one CTA's run.  A segment that is not the whole item leaves
// unnormalised sums, row maxima and row sums in the workspace, and the join
// kernel adds the parts in order.  The split depends on the lengths and the SM
// count alone, so the same call gives the same bits.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "s2_common.cuh"
#include "s2_ptx.cuh"

namespace s2 {
namespace cache {

constexpr float kFloor = -3.0e38f;  // running maximum of a row that has seen no key (finite: no inf - inf)

// The lengths of request i, and its units.
struct Req {
  int ctx, n, row0;  // cached tokens, new tokens, first row of q
  int keys;          // keys in all
  int kt, ni;        // key tiles, items a kv head
  long long units;   // Hkv * ni * kt
};
// KEYS: keys of a tile; tokens: new tokens of an item.
template <int KEYS>
__device__ __forceinline__ Req request(const CacheAttnArgs& a, int i, int tokens) {
  Req r;
  const int c0 = a.cu_seqlens[i], c1 = a.cu_seqlens[i + 1], cl = a.ctx_lens[i];
  r.row0 = min(max(c0, 0), a.T);
  r.n = min(max(c1, r.row0), a.T) - r.row0;
  const long long most = static_cast<long long>(a.max_blocks) << a.bs_log2;  // places the table has
  r.ctx = static_cast<int>(min(static_cast<long long>(max(cl, 0)), most));
  r.keys = static_cast<int>(min(static_cast<long long>(r.ctx) + r.n, most));
  r.kt = (r.keys + KEYS - 1) / KEYS;
  r.ni = (r.n + tokens - 1) / tokens;
  r.units = static_cast<long long>(a.Hkv) * r.ni * r.kt;
  return r;
}

struct Seg {
  int ri, kvh;
  int row0, ctx, keys;  // the request (row0: first row of q)
  int tok, ntok;        // first new token of the item in the request, and their number
  int kt0, tiles;       // first key tile, key tiles to work on (0: none is visible, -1: no more segments)
  int whole, first;     // the whole item; the part with key tile 0
  int last_cta;         // first && !whole: CTA with the item's last part
};

// A CTA's run of units and the walk through its segments.
struct Run {
  long long u0, u1, rbase, per;  // units left; first unit of request ri; units of a run
  int ri;
};

// Finds the run of this CTA and the request it begins in; false if it has no
// units.  All THREADS threads of the block call it; `sums` and `found` are
// shared memory.
template <int THREADS, int KEYS>
__device__ __forceinline__ bool locate(const CacheAttnArgs& a, int tokens, int min_units, long long* sums,
                                       long long* found, Run& run) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // exclusive prefix of v over the block, and the block's sum
  auto scan = [&](long long v, long long& all) {
    long long inc = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, m);
      if (lane >= m) inc += o;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    long long base = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) base += sums[w];
      all += sums[w];
    }
    return base + inc - v;
  };
  long long total = 0, mine = 0, at = 0;
  for (int base = 0; base < a.R; base += THREADS) {
    long long all;
    mine = base + tid < a.R ? request<KEYS>(a, base + tid, tokens).units : 0;
    at = total + scan(mine, all);
    total += all;
  }
  run.per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(min_units));
  run.u0 = run.per * blockIdx.x;
  run.u1 = min(run.u0 + run.per, total);
  if (run.u0 >= run.u1) return false;
  long long before = 0;
  for (int base = 0; base < a.R; base += THREADS) {
    if (a.R > THREADS) {  // one chunk: its scan is still there
      long long all;
      mine = base + tid < a.R ? request<KEYS>(a, base + tid, tokens).units : 0;
      at = before + scan(mine, all);
      before += all;
    }
    if (run.u0 >= at && run.u0 < at + mine) {
      found[0] = base + tid;
      found[1] = at;
    }
    if (a.R > THREADS && run.u0 < before) break;  // uniform
  }
  __syncthreads();
  run.ri = static_cast<int>(found[0]);
  run.rbase = found[1];
  return true;
}

template <int KEYS>
__device__ __forceinline__ bool next_segment(const CacheAttnArgs& a, int tokens, Run& w, Seg& s) {
  while (w.u0 < w.u1) {
    const Req r = request<KEYS>(a, w.ri, tokens);
    if (w.u0 >= w.rbase + r.units) {
      w.rbase += r.units;
      ++w.ri;
      continue;
    }
    const long long in = w.u0 - w.rbase, item = in / r.kt;  // item = kvh * ni + item of the kv head
    const int e = static_cast<int>(item % r.ni);
    s.ri = w.ri;
    s.kvh = static_cast<int>(item / r.ni);
    s.row0 = r.row0;
    s.ctx = r.ctx;
    s.keys = r.keys;
    s.tok = e * tokens;
    s.ntok = min(tokens, r.n - s.tok);
    s.kt0 = static_cast<int>(in - item * r.kt);
    const int kt1 = static_cast<int>(min(static_cast<long long>(r.kt), s.kt0 + (w.u1 - w.u0)));
    // chains: keys behind the item's last token are not visited
    const int reach = a.mask != nullptr ? r.keys : min(r.ctx + min(s.tok + s.ntok, r.keys - r.ctx), r.keys);
    s.tiles = max(min(kt1, (reach + KEYS - 1) / KEYS) - s.kt0, 0);
    s.first = s.kt0 == 0;
    s.whole = s.first && kt1 == r.kt;
    s.last_cta = static_cast<int>((w.rbase + (item + 1) * r.kt - 1) / w.per);
    w.u0 += kt1 - s.kt0;
    return true;
  }
  return false;
}

// The drafts a row sees, as bits: its mask without the bits of drafts that do not exist.
__device__ __forceinline__ unsigned long long visible_drafts(const CacheAttnArgs& a, const Seg& s, int token) {
  const int drafts = s.keys - s.ctx;
  return a.mask[token] & (drafts >= 64 ? ~0ull : (1ull << drafts) - 1ull);
}

__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? neg_inf() : (m + log2f(l)) * 0.69314718055994531f;
}

// A part in the workspace: ROWS x D sums, then ROWS maxima (log2 units) and
// ROWS sums.  CTA c's slot 1 holds the part of the item that begins in it,
// slot 0 the part of an item that began before.
template <int ROWS, int D>
struct Part {
  static constexpr size_t kFloats = static_cast<size_t>(ROWS) * (D + 2);
  static __device__ __forceinline__ float* at(const CacheAttnArgs& a, int cta, int slot) {
    return a.partial + (2 * static_cast<size_t>(cta) + slot) * kFloats;
  }
};

// Lets the dependent launch begin (its blocks wait for this grid's end where
// they need its results), and that wait.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Joins the parts of the item that begins in CTA blockIdx.x and runs on: block
// y its rows 8 y .. 8 y + 7.  With few parts each of the 8 warps joins a row,
// with many all of them share a row's parts.  A part whose row saw no key has
// l = 0 and nothing else in it.  TILE: rows of a row tile (its first a.tpt
// tokens); the launch overlaps the attention kernel's end.
template <int ROWS, int TILE, int KEYS, int D>
__global__ void __launch_bounds__(256) s2_cache_join_kernel(CacheAttnArgs a, int tokens) {
  constexpr int PER = D / 32;  // columns a lane
  __shared__ float share[8][D + 1];
  wait_for_primary();
  const int4 d = a.desc[blockIdx.x];
  if (d.x < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kvh = d.y, tok0 = d.z, first = blockIdx.x, parts = d.w - first + 1;
  const Req r = request<KEYS>(a, d.x, tokens);
  const int share_of = parts > 8 ? 8 : 1, sub = parts > 8 ? warp : 0;
  for (int row = blockIdx.y * 8 + (parts > 8 ? 0 : warp); row < blockIdx.y * 8 + 8; row += parts > 8 ? 1 : 8) {
    const int tile = row / TILE, in = row - tile * TILE, jt = in / a.rep, tok = tok0 + tile * a.tpt + jt;
    if (jt >= a.tpt || tok >= r.n) continue;  // uniform in the warps that share the row
    auto part = [&](int p) { return Part<ROWS, D>::at(a, first + p, p == 0 ? 1 : 0); };
    float m = kFloor;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, part(p)[ROWS * D + row]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    float l = 0.f, acc[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[k] = 0.f;
    for (int p0 = sub; p0 < parts; p0 += 32 * share_of) {  // this warp's next 32 parts: a lane each for their statistics
      const int mine = p0 + lane * share_of;
      const float lp = mine < parts ? part(mine)[ROWS * (D + 1) + row] : 0.f;
      const float f = lp != 0.f ? ex2_approx(part(mine)[ROWS * D + row] - m) : 0.f;
      const int n = min(32, (parts - p0 + share_of - 1) / share_of);
#pragma unroll 4
      for (int x = 0; x < n; ++x) {
        const float lx = __shfl_sync(0xffffffffu, lp, x), fx = __shfl_sync(0xffffffffu, f, x);
        if (lx != 0.f) {
          const float* src = part(p0 + x * share_of) + row * D + lane * PER;
          l = fmaf(fx, lx, l);
          if constexpr (PER == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            acc[0] = fmaf(fx, v.x, acc[0]);
            acc[1] = fmaf(fx, v.y, acc[1]);
            acc[2] = fmaf(fx, v.z, acc[2]);
            acc[3] = fmaf(fx, v.w, acc[3]);
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            acc[0] = fmaf(fx, v.x, acc[0]);
            acc[1] = fmaf(fx, v.y, acc[1]);
          }
        }
      }
    }
    if (parts > 8) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < PER; ++k) share[warp][lane * PER + k] = acc[k];
      if (lane == 0) share[warp][D] = l;
      __syncthreads();
      if (warp > 0) continue;
#pragma unroll
      for (int w = 1; w < 8; ++w) {
        l += share[w][D];
#pragma unroll
        for (int k = 0; k < PER; ++k) acc[k] += share[w][lane * PER + k];
      }
    }
    const int h = kvh * a.rep + in - jt * a.rep, tk = r.row0 + tok;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.o + (static_cast<size_t>(tk) * a.H + h) * D + lane * PER);
#pragma unroll
    for (int k = 0; k < PER / 2; ++k) out[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    if (lane == 0) a.lse[static_cast<size_t>(h) * a.T + tk] = lse_of(m, l);
  }
}

// The join as a dependent launch of the attention kernel before it in the stream.
template <int ROWS, int TILE, int KEYS, int D>
cudaError_t launch_join(const CacheAttnArgs& a, int tokens, int grid, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, ROWS / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  prof_before(stream, kKernelCacheMerge);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, s2_cache_join_kernel<ROWS, TILE, KEYS, D>, a, tokens);
  prof_after(stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace cache
}  // namespace s2
