// What the two cache attention kernels (s2_cache_dec.cu, s2_cache_tc.cu) share:
// the numbering of the work and its split over the CTAs, and the join of items
// that more than one CTA worked on.
//
// An item is the new tokens of one row tile (or pair of tiles) of one (request,
// kv head) against all of the request's keys; a unit is one key tile of an
// item.  All units of a batch are numbered request by request and dealt to the
// CTAs in equal contiguous runs, so that a batch of very different lengths, or
// one long request, loads every SM alike -- where tokens see (nearly) all of their
// request's keys.  Units that a chain's earlier tokens do not see are counted
// and cost nothing, so for a long prompt the runs are not alike: by the same
// numbering, the busiest has 1.86 times the mean of a prompt of 4096 tokens (32/8
// heads, no context; 494 us), 1.80 of 1024 (64/8), 1.29 of 4096 over 4096 (739 us).
// `side` CTAs in a row work side by side: each takes the same run of another kv
// head, so that what they read at a time lies together in the cache (64 requests
// of 333 to 16384 keys, 8 kv heads: 337 us so, 340 one head after the other).  A
// segment is the part of an item that lies in one CTA's run.  A segment that is
// not the whole item leaves unnormalised sums, row maxima and row sums in the
// workspace, and the join kernel adds the parts in order.  The split depends on
// the lengths and the SM count alone, so the same call gives the same bits.
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
  long long units;   // Hkv / side * ni * kt
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
  r.units = static_cast<long long>(a.Hkv / a.side) * r.ni * r.kt;
  return r;
}

// Keys that the request's first `tokens` new tokens see at most (chains: up to
// the last one's own).
__device__ __forceinline__ int visible_keys(const CacheAttnArgs& a, const Req& r, int tokens) {
  return a.mask != nullptr ? r.keys : min(r.ctx + min(tokens, r.keys - r.ctx), r.keys);
}

// Debug build: row (token tk, query head) lies in o and lse.
__device__ __forceinline__ bool row_in(const CacheAttnArgs& a, int tk, int head, uint32_t where) {
  return in_bounds(a.status, tk, a.T, where) && in_bounds(a.status, head, a.H, where);
}

// The block of request i's key, -1 where the debug build finds the entry outside the table.
__device__ __forceinline__ int block_of(const CacheAttnArgs& a, int i, int key) {
  const int col = key >> a.bs_log2;
  if (!in_bounds(a.status, i, a.R, 740) || !in_bounds(a.status, col, a.max_blocks, 741)) return -1;
  return a.block_tables[static_cast<size_t>(i) * a.max_blocks + col];
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
  Req r;                         // request ri (ri < R)
};
// What the CTA's threads share while they look for its first request.
struct Found {
  long long rbase;
  int ri;
  Req r;
};

// Finds the run of this CTA and the request it begins in; false if it has no
// units.  All THREADS threads of the block call it; `sums` and `found` are
// shared memory.  (The first request comes out of it as it was scanned: reading
// it again would cost every CTA's first load another trip to L2.)
template <int THREADS, int KEYS>
__device__ __forceinline__ bool locate(const CacheAttnArgs& a, int tokens, int min_units, long long* sums,
                                       Found* found, Run& run) {
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
  Req r = {};
  for (int base = 0; base < a.R; base += THREADS) {
    long long all;
    if (base + tid < a.R) r = request<KEYS>(a, base + tid, tokens);
    mine = base + tid < a.R ? r.units : 0;
    at = total + scan(mine, all);
    total += all;
  }
  const int runs = gridDim.x / a.side;
  run.per = max((total + runs - 1) / runs, static_cast<long long>(min_units));
  run.u0 = run.per * (blockIdx.x / a.side);
  run.u1 = min(run.u0 + run.per, total);
  if (run.u0 >= run.u1) return false;
  if (tid == 0) found->ri = a.R;
  __syncthreads();
  long long before = 0;
  for (int base = 0; base < a.R; base += THREADS) {
    if (a.R > THREADS) {  // one chunk: its scan is still there
      long long all;
      if (base + tid < a.R) r = request<KEYS>(a, base + tid, tokens);
      mine = base + tid < a.R ? r.units : 0;
      at = before + scan(mine, all);
      before += all;
    }
    if (run.u0 >= at && run.u0 < at + mine) {
      found->ri = base + tid;
      found->rbase = at;
      found->r = r;
    }
    if (a.R > THREADS && run.u0 < before) break;  // uniform
  }
  __syncthreads();
  run.ri = found->ri;
  run.rbase = found->rbase;
  run.r = found->r;
  return true;
}

// The next segment of the run; false at its end.  Called by a whole warp with the
// same arguments: its lanes look for the next request with new tokens together.
template <int KEYS>
__device__ __forceinline__ bool next_segment(const CacheAttnArgs& a, int tokens, Run& w, Seg& s) {
  while (w.u0 < w.u1 && w.ri < a.R) {  // (the second holds unless lengths change under the kernel)
    const Req& r = w.r;
    if (w.u0 >= w.rbase + r.units) {
      w.rbase += r.units;
      for (++w.ri; w.ri < a.R; w.ri += 32) {
        const int i = w.ri + (threadIdx.x & 31);
        const unsigned busy = __ballot_sync(0xffffffffu, i < a.R && request<KEYS>(a, i, tokens).units > 0);
        if (busy != 0) {
          w.ri += __ffs(busy) - 1;
          w.r = request<KEYS>(a, w.ri, tokens);
          break;
        }
      }
      continue;
    }
    const long long in = w.u0 - w.rbase, item = in / r.kt;  // item = kvh / side * ni + item of the kv head
    const int e = static_cast<int>(item % r.ni), mate = blockIdx.x % a.side;
    s.ri = w.ri;
    s.kvh = static_cast<int>(item / r.ni) * a.side + mate;
    s.row0 = r.row0;
    s.ctx = r.ctx;
    s.keys = r.keys;
    s.tok = e * tokens;
    s.ntok = min(tokens, r.n - s.tok);
    s.kt0 = static_cast<int>(in - item * r.kt);
    const int kt1 = static_cast<int>(min(static_cast<long long>(r.kt), s.kt0 + (w.u1 - w.u0)));
    s.tiles = max(min(kt1, (visible_keys(a, r, s.tok + s.ntok) + KEYS - 1) / KEYS) - s.kt0, 0);
    s.first = s.kt0 == 0;
    s.whole = s.first && kt1 == r.kt;
    s.last_cta = static_cast<int>((w.rbase + (item + 1) * r.kt - 1) / w.per) * a.side + mate;
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

// Whether one of two / eight bf16 values is infinite or NaN (all exponent bits set).
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ bool nonfinite8(const uint4& u) {
  return nonfinite2(u.x) || nonfinite2(u.y) || nonfinite2(u.z) || nonfinite2(u.w);
}

__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? neg_inf() : (m + log2f(l)) * 0.69314718055994531f;
}

// acc (bit patterns, 32 columns from c0 of one row) out: o normalised, or the partial as it is.
__device__ __forceinline__ void store_o32(__nv_bfloat16* o, float* part, bool whole, const uint32_t (&v)[32], float inv) {
  if (whole) {
    store_row32(o, v, inv);
  } else {
    uint4* p = reinterpret_cast<uint4*>(part);
#pragma unroll
    for (int q = 0; q < 8; ++q) p[q] = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  }
}

// Adds the infinite and NaN values of V in the segment's drafts to the stored
// row (o, or its part) of a token that sees them; any weight turns such a value
// into itself.  Out of line: such values are an error of the model's.
template <int D>
__device__ __noinline__ void add_odd(const CacheAttnArgs& a, const Seg& sg, int token, __nv_bfloat16* o, float* part) {
  const int j_tok = token - sg.row0, last = min((sg.kt0 + sg.tiles) * kTile, sg.keys);
  const unsigned long long see = a.mask != nullptr ? visible_drafts(a, sg, token) : 0ull;
  for (int key = max(sg.kt0 * kTile, sg.ctx); key < last; ++key) {
    const int d = key - sg.ctx, blk = block_of(a, sg.ri, key);
    if (a.mask != nullptr ? d >= 64 || !(see >> d & 1) : d > j_tok) continue;
    if (blk < 0 || blk >= a.num_blocks) continue;
    const size_t place = (static_cast<size_t>(blk) << a.bs_log2) + (key & ((1 << a.bs_log2) - 1));
    const __nv_bfloat16* src = a.v_cache + (place * a.Hkv + sg.kvh) * D;
    for (int i = 0; i < D; ++i) {
      const float x = __bfloat162float(src[i]);
      if (isfinite(x)) continue;
      if (sg.whole)
        o[i] = __float2bfloat16(__bfloat162float(o[i]) + x);
      else
        part[i] += x;
    }
  }
}

// Makes a landed V tile (128-byte-swizzled 64-column slabs of kTile rows) safe
// for the product; the 128 threads of a warpgroup call it, `row` 0 .. 127.  Rows
// behind the last key (`valid` rows hold keys) within its 16-key step are zeroed:
// stale cache rows may hold anything.  So are infinite and NaN values of the
// tile's drafts (its last `drafts` keys), which a product would add as 0 V to
// rows that do not see them; `odd` is set, and add_odd adds them to the rows that
// do.
template <int D>
__device__ __forceinline__ void clean_v(uint32_t tile, int valid, int drafts, int row, uint32_t& odd) {
  const int rows = drafts + (-valid & 15);
  for (int e = row; e < rows * (D / 8); e += 128) {
    const int r = valid - drafts + e / (D / 8), c = e % (D / 8);
    const uint32_t at = tile + (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (r < valid) {
      w = lds_u4(at);
      if (!nonfinite8(w)) continue;
      odd = 1;
      uint32_t* h = &w.x;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if ((h[x] & 0x7f80u) == 0x7f80u) h[x] &= 0xffff0000u;
        if ((h[x] & 0x7f800000u) == 0x7f800000u) h[x] &= 0xffffu;
      }
    }
    st_shared_v4(at, w.x, w.y, w.z, w.w);
  }
  fence_proxy_async_smem();
}

// Scores of one row against the 128 keys from key0: -inf where the row's token
// (the j_tok-th new one of the request) does not see the key.
__device__ __forceinline__ void mask_row128(const CacheAttnArgs& a, const Seg& s, int key0, int j_tok,
                                            uint32_t (&sr)[4][32]) {
  if (a.mask == nullptr) {
    const int lim = min(s.ctx + j_tok, s.keys - 1) - key0;  // last visible column
#pragma unroll
    for (int c = 0; c < 128; ++c)
      if (c > lim) sr[c >> 5][c & 31] = __float_as_uint(neg_inf());
  } else {
    // visible columns as 4 words: cached keys, then the draft bits (of the request's rows)
    const unsigned long long see = j_tok < s.tok + s.ntok ? visible_drafts(a, s, s.row0 + j_tok) : 0ull;
    const int d0 = s.ctx - key0;  // column of draft 0 (below 0: drafts begin in an earlier tile)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int at = d0 - 32 * w;  // draft 0 relative to this word
      uint32_t bits;
      if (at >= 32)
        bits = 0xffffffffu;
      else if (at > 0)
        bits = ((1u << at) - 1u) | static_cast<uint32_t>(see << at);
      else
        bits = at > -64 ? static_cast<uint32_t>(see >> -at) : 0u;
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (!(bits >> c & 1u)) sr[w][c] = __float_as_uint(neg_inf());
    }
  }
}

// A part in the workspace: ROWS x D sums, then ROWS maxima (log2 units) and
// ROWS sums.  CTA c's slot 1 holds the part of the item that begins in it,
// slot 0 the part of an item that began before.
template <int ROWS, int D>
struct Part {
  static constexpr size_t kFloats = static_cast<size_t>(ROWS) * (D + 2);
  static __device__ __forceinline__ float* at(const CacheAttnArgs& a, int cta, int slot) {
    const size_t off = (2 * static_cast<size_t>(cta) + slot) * kFloats;
    return a.partial + (in_bounds(a.status, off + kFloats - 1, kCachePartFloats<D>, 742) ? off : 0);
  }
};

// The join work of CTA blockIdx.x: an item that begins in it and runs on.
__device__ __forceinline__ int4 join_work(const Seg& s) {
  return make_int4(s.row0 + s.tok, s.ntok, s.kvh, s.last_cta);
}

// Joins the parts of the item that begins in CTA blockIdx.x and runs on.  WPR
// warps share a row and take every WPR-th part (few rows, many parts: the
// few-row kernel), or a warp joins RPW rows side by side (many rows, few parts).
// A part whose row saw no key has l = 0 and may hold anything else: its sums are
// loaded all the same, so that no load waits for another, and left out.  TILE:
// rows of a row tile (its first a.tpt tokens).  The launch overlaps the
// attention kernel's end.
template <int ROWS, int TILE, int D, int WPR, int RPW>
__global__ void __launch_bounds__(256) s2_cache_join_kernel(CacheAttnArgs a) {
  constexpr int PER = D / 32;  // columns a lane
  __shared__ float share[8][D + 1];
  wait_for_primary();
  const int4 d = a.desc[blockIdx.x];
  if (d.y < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPR;
  const int first = blockIdx.x, parts = (d.w - first) / a.side + 1;
  const int row0 = (blockIdx.y * (8 / WPR) + warp / WPR) * RPW;
  const int lead = WPR == 1 ? row0 : blockIdx.y * (8 / WPR) * RPW;  // warps that share rows leave together
  if ((lead / TILE) * a.tpt + (lead % TILE) / a.rep >= d.y) return;  // rows behind the item's
  auto part = [&](int p) { return Part<ROWS, D>::at(a, first + p * a.side, p == 0 ? 1 : 0); };
  float m[RPW], l[RPW], acc[RPW][PER];
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    m[i] = kFloor;
    l[i] = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[i][k] = 0.f;
  }
  // 32 parts of this warp at a time, a lane each for their statistics
  for (int p0 = sub; p0 < parts; p0 += 32 * WPR) {
    const int p = p0 + WPR * lane, n = min(32, (parts - p0 + WPR - 1) / WPR);
    float lp[RPW], f[RPW];
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      lp[i] = p < parts ? part(p)[ROWS * (D + 1) + row0 + i] : 0.f;
      f[i] = p < parts ? part(p)[ROWS * D + row0 + i] : kFloor;
    }
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      float mx = lp[i] != 0.f ? f[i] : kFloor;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
      mx = fmaxf(mx, m[i]);
      const float old = ex2_approx(m[i] - mx);  // the parts before: 1 unless there are more than 32
      m[i] = mx;
      l[i] *= old;
#pragma unroll
      for (int k = 0; k < PER; ++k) acc[i][k] *= old;
      f[i] = lp[i] != 0.f ? ex2_approx(f[i] - mx) : 0.f;
    }
#pragma unroll 4
    for (int x = 0; x < n; ++x) {
      const float* src = part(p0 + WPR * x) + row0 * D + lane * PER;
      float v[RPW][PER];
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        if constexpr (PER == 4)
          *reinterpret_cast<float4*>(v[i]) = *reinterpret_cast<const float4*>(src + i * D);
        else
          *reinterpret_cast<float2*>(v[i]) = *reinterpret_cast<const float2*>(src + i * D);
      }
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        const float lx = __shfl_sync(0xffffffffu, lp[i], x), fx = __shfl_sync(0xffffffffu, f[i], x);
        if (lx == 0.f) continue;
        l[i] = fmaf(fx, lx, l[i]);
#pragma unroll
        for (int k = 0; k < PER; ++k) acc[i][k] = fmaf(fx, v[i][k], acc[i][k]);
      }
    }
  }
  if constexpr (WPR > 1) {
    static_assert(RPW == 1, "warps that share a row join one");
    __shared__ float share_m[8];
#pragma unroll
    for (int k = 0; k < PER; ++k) share[warp][lane * PER + k] = acc[0][k];
    if (lane == 0) {
      share[warp][D] = l[0];
      share_m[warp] = m[0];
    }
    __syncthreads();
    if (sub > 0) return;
    float mx = m[0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) mx = fmaxf(mx, share_m[warp + w]);
    const float own = ex2_approx(m[0] - mx);
    m[0] = mx;
    l[0] *= own;
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[0][k] *= own;
#pragma unroll
    for (int w = 1; w < WPR; ++w) {
      const float fw = ex2_approx(share_m[warp + w] - mx);
      l[0] = fmaf(fw, share[warp + w][D], l[0]);
#pragma unroll
      for (int k = 0; k < PER; ++k) acc[0][k] = fmaf(fw, share[warp + w][lane * PER + k], acc[0][k]);
    }
  }
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    const int tile = (row0 + i) / TILE, in = row0 + i - tile * TILE, jt = in / a.rep, tok = tile * a.tpt + jt;
    if (jt >= a.tpt || tok >= d.y) continue;  // a row of no token
    const int tk = d.x + tok, head = d.z * a.rep + in - jt * a.rep;
    if (!row_in(a, tk, head, 743)) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    uint32_t* out = reinterpret_cast<uint32_t*>(a.o + (static_cast<size_t>(tk) * a.H + head) * D + lane * PER);
#pragma unroll
    for (int k = 0; k < PER / 2; ++k) out[k] = pack_bf16x2(acc[i][2 * k] * inv, acc[i][2 * k + 1] * inv);
    if (lane == 0) a.lse[static_cast<size_t>(head) * a.T + tk] = lse_of(m[i], l[i]);
  }
}

// The join as a dependent launch of the attention kernel before it in the stream.
template <int ROWS, int TILE, int D, int WPR, int RPW>
cudaError_t launch_join(const CacheAttnArgs& a, int grid, cudaStream_t stream) {
  prof_before(stream, kKernelCacheMerge);
  // rows that an item can have, in blocks of 8 / WPR * RPW
  const int most = ROWS == TILE && a.T < a.tpt ? a.T * a.rep : ROWS, per = 8 / WPR * RPW;
  const cudaError_t e = launch_dependent(s2_cache_join_kernel<ROWS, TILE, D, WPR, RPW>,
                                         dim3(grid, (most + per - 1) / per), 256, stream, a);
  prof_after(stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace cache
}  // namespace s2
