// Attention of few new tokens over a paged cache: decoding, and short chains or
// trees of drafts (at most 16 rows of (token, head) share a kv head's keys in a
// tile).  The same operation as s2_cache_tc.cu, for calls that reading the
// cache bounds: with one row in 16 or 4 in 128 the tensor work is small
// whatever unit does it, and what counts is that loads never stop.
//
// Rows.  The rep = H/Hkv <= 16 query heads of a kv head form one 16-row tile
// with floor(16 / rep) tokens: row = token * rep + head in group, the order a
// {64 columns, rep heads, tokens} TMA box lands in shared memory.
//
// Two CTAs an SM, each a TMA producer warp and four consumer warps.  The
// producer walks the CTA's segments on its own, through a ring of 64-key stages
// (K and V, 32 KB at head dim 128: 6 stages an SM, 192 KB in flight where some
// 45 KB cover the latency at full bandwidth), and hands each segment's
// description and query rows over in a three-slot ring, so that no load waits for
// arithmetic and the stages keep filling across segments.  A consumer warp
// takes 16 of a stage's 64 keys through mma.sync with its own running maximum
// and sum (fp32): no synchronisation inside a segment but the stages' own
// barriers.  At its end the four warps join through the last stage's memory, after
// one meeting.  P is rounded to bf16 for the product with V, its sums are taken
// before.
//
// A call with few items and short tables takes a form of its own (the host's rule
// has the figures): a cluster of CTAs an item, joined through distributed shared
// memory.
//
// Measured, head dim 128 (bf16): 64 requests of 333 to 16384 keys, 32/8 heads,
// 335 to 339 us, 6.6 TB/s, what a copy reaches; one request of 4097 keys, 32/8
// heads, 12.6 us, 10.9 of it on the GPU (some 2 to 4 more without clusters):
// latency.
//
// Rows of V behind the last key may hold anything (stale cache rows): the
// fragments that hold them are zeroed in registers.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "s2_cache.cuh"

namespace s2 {

namespace {

using namespace cache;

constexpr int kRows = kCacheRows;  // rows of a tile
constexpr int kKeys = 64;          // keys of a stage
constexpr int kWarps = 4;          // consumers
constexpr int kDecThreads = 32 * (kWarps + 1);

template <int D>
struct DecCfg {
  static constexpr int NS = D == 128 ? 3 : 6;       // stages
  static constexpr int NQ = 3;                      // segments handed over
  static constexpr int SLAB = kKeys * 128;          // one 64-column slab of a stage's K or V
  static constexpr int TILE = kKeys * D * 2;        // K or V
  static constexpr int STAGE = 2 * TILE;
  static constexpr int QSLAB = kRows * 128;
  static constexpr int QSLOT = kRows * D * 2;
  static constexpr int OFF_Q = NS * STAGE;
  static constexpr int SMEM = OFF_Q + NQ * QSLOT + 1024;
  static_assert(kWarps * kRows * D * 4 == STAGE, "the warps' sums fit the rows of their keys");
  static_assert(2 * (SMEM + 2048) <= 233472, "two CTAs an SM");
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Address of 16-byte chunk c of row r in slabs of `slab` bytes written by TMA
// with the 128-byte swizzle (slabs 1024-byte aligned).
__device__ __forceinline__ uint32_t swz(uint32_t base, int slab, int r, int c) {
  return base + (c >> 3) * slab + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster that have not ended meet; what was written to
// shared memory before is visible in the cluster after.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address of `addr` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_peer_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_peer_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// The request and the new tokens of row tile `at`, the requests' row tiles being
// counted in order; false if there are fewer.  Each warp looks for itself.
__device__ __forceinline__ bool find_item(const CacheAttnArgs& a, int at, Req& r, Seg& s) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < a.R; base += 32) {
    Req mine = {};
    if (base + lane < a.R) mine = request<kKeys>(a, base + lane, a.tpt);
    int end = mine.ni;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, end, m);
      if (lane >= m) end += o;
    }
    const unsigned past = __ballot_sync(0xffffffffu, at < end);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      s.ri = base + l;
      s.row0 = r.row0 = __shfl_sync(0xffffffffu, mine.row0, l);
      s.ctx = r.ctx = __shfl_sync(0xffffffffu, mine.ctx, l);
      s.keys = r.keys = __shfl_sync(0xffffffffu, mine.keys, l);
      s.tok = (at - __shfl_sync(0xffffffffu, end - mine.ni, l)) * a.tpt;
      s.ntok = min(a.tpt, __shfl_sync(0xffffffffu, mine.n, l) - s.tok);
      return true;
    }
    at -= __shfl_sync(0xffffffffu, end, 31);
  }
  return false;
}

// Waits (bounded) for the last fill of every slot of a ring.  Out of line, away from what a small call has to
// fetch (one token over 4097 keys: 12.6 us a call, 13.0 in line).
__device__ __noinline__ void drain_ring(uint32_t bars, int slots, int fills) {
  for (int s = 0; s < slots && s < fills; ++s) drain_wait(bars + 8 * s, ((fills - 1 - s) / slots) & 1);
}

// CL: the form for few items.  Each gets a cluster of CTAs (one or more) with an
// equal share of its key tiles, which joins its parts through distributed shared
// memory: one launch, no table of work and nothing in the workspace.
template <int D, bool CL>
__global__ void __launch_bounds__(kDecThreads, 2)
    s2_cache_dec_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const CacheAttnArgs a) {
  using C = DecCfg<D>;
  constexpr int NS = C::NS, NQ = C::NQ;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t bar_full[NS], bar_empty[NS], bar_qfull[NQ], bar_qempty[NQ], bar_join;
  __shared__ uint32_t abort_flag;
  __shared__ long long sums[kDecThreads / 32];
  __shared__ Found found;
  __shared__ Seg segs[NQ];
  __shared__ float2 stats[2][kWarps][kRows];  // row maxima and sums of the warps, by turns
  __shared__ float2 part_stats[kRows];        // CL: the part's row maxima and sums
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < 3) tma_prefetch_desc(tid == 0 ? &tmQ : tid == 1 ? &tmK : &tmV);
  Run run;
  Seg only;  // CL: this CTA's share of its cluster's item
  if constexpr (CL) {
    const int item = blockIdx.x / cluster_size(), share = cluster_rank();
    Req r;
    if (!find_item(a, item / a.Hkv, r, only)) return;  // the whole cluster
    only.kvh = item % a.Hkv;
    const int tiles = (visible_keys(a, r, only.tok + only.ntok) + kKeys - 1) / kKeys;
    const int per = (tiles + cluster_size() - 1) / cluster_size();
    only.kt0 = share * per;
    only.tiles = max(min(per, tiles - only.kt0), 0);
    only.whole = only.first = only.last_cta = 0;
  } else {
    launch_dependents();
    if (tid == 0) a.desc[blockIdx.x] = make_int4(0, -1, 0, 0);
    if (!locate<kDecThreads, kKeys>(a, a.tpt, kCacheMinUnits, sums, &found, run)) return;
  }
  const uint32_t sbase = smem_u32(smem);
  WaitCtx wc{&abort_flag, a.status, a.wait_limit_ns};
  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);
      mbar_init(smem_u32(&bar_empty[s]), kWarps);
    }
    for (int s = 0; s < NQ; ++s) {
      mbar_init(smem_u32(&bar_qfull[s]), 1);
      mbar_init(smem_u32(&bar_qempty[s]), kWarps);
    }
    mbar_init(smem_u32(&bar_join), kWarps);
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    int L = 0, qu = 0;
    bool ok = true;
    const int page_log2 = min(a.bs_log2, 6), page_rows = 1 << page_log2;
    Seg sg;
    for (;;) {
      bool more;
      if constexpr (CL) {
        more = qu == 0;
        sg = only;
      } else {
        more = next_segment<kKeys>(a, a.tpt, run, sg);
      }
      const int qs = qu % NQ;
      if (qu >= NQ && !(ok = warp_wait(smem_u32(&bar_qempty[qs]), (qu / NQ - 1) & 1, wc, 140))) break;
      if (lane == 0) {
        if (!more) sg.tiles = -1;
        segs[qs] = sg;
        if (more && sg.tiles > 0) {
          mbar_arrive_expect_tx(smem_u32(&bar_qfull[qs]), a.tpt * a.rep * 128 * (D / 64));
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sbase + C::OFF_Q + qs * C::QSLOT + c * C::QSLAB, &tmQ, smem_u32(&bar_qfull[qs]), c * 64,
                        sg.kvh * a.rep, in_bounds(a.status, sg.row0 + sg.tok, a.T, 744) ? sg.row0 + sg.tok : 0, 0);
        } else {
          mbar_arrive(smem_u32(&bar_qfull[qs]));
        }
      }
      __syncwarp();
      ++qu;
      if (!more) break;
      for (int i = 0; ok && i < sg.tiles; ++i) {
        const int key = (sg.kt0 + i) * kKeys + (lane << page_log2);
        const bool mine = lane < (kKeys >> page_log2) && key < sg.keys;
        int row = 0;  // a block outside the cache reads as zeros: its row lies behind the tensor
        if (mine) {
          const int blk = block_of(a, sg.ri, key);
          row = data_in_range(a.status, blk, a.num_blocks, 711) ? (blk << a.bs_log2) + (key & ((1 << a.bs_log2) - 1))
                                                                : a.num_blocks << a.bs_log2;
        }
        const int s = L % NS, r = L / NS, pages = __popc(__ballot_sync(0xffffffffu, mine));
        if (r > 0 && !(ok = warp_wait(smem_u32(&bar_empty[s]), (r - 1) & 1, wc, 141))) break;
        if (lane == 0) mbar_arrive_expect_tx(smem_u32(&bar_full[s]), 2 * pages * page_rows * 128 * (D / 64));
        __syncwarp();
        if (mine)
          for (int c = 0; c < D / 64; ++c) {
            const uint32_t dst = sbase + s * C::STAGE + c * C::SLAB + (lane << page_log2) * 128;
            tma_load_4d(dst, &tmK, smem_u32(&bar_full[s]), c * 64, sg.kvh, row, 0);
            tma_load_4d(dst + C::TILE, &tmV, smem_u32(&bar_full[s]), c * 64, sg.kvh, row, 0);
          }
        __syncwarp();
        ++L;
      }
      if (!ok) break;
    }
    if ((!CL || *wc.abort) && lane == 0) {
      // never leave copies in flight into shared memory, whether or not a
      // consumer has given up by now: it can do so after this warp's last copy
      // (in clusters that is asked after the meeting, off the way of small calls)
      drain_ring(smem_u32(bar_qfull), NQ, qu);
      drain_ring(smem_u32(bar_full), NS, L);
    }
  } else {
    // ------------------------------------------------------------ consumers
    const float sl2 = a.scale_log2;
    int L = 0, nj = 0;
    // the four warps meet (a bounded wait, where a named barrier would block for
    // good once a warp has given up)
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_join));
      return warp_wait(smem_u32(&bar_join), nj++ & 1, wc, 144);
    };
    for (int qu = 0;; ++qu) {
      const int qs = qu % NQ;
      if (!warp_wait(smem_u32(&bar_qfull[qs]), (qu / NQ) & 1, wc, 142)) break;
      const Seg sg = segs[qs];
      if (sg.tiles < 0) break;
      const uint32_t sq = sbase + C::OFF_Q + qs * C::QSLOT;
      const int rows = sg.ntok * a.rep;
      float o[D / 8][4];
#pragma unroll
      for (int d = 0; d < D / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
      float m[2] = {kFloor, kFloor}, l[2] = {0.f, 0.f};
      bool ok = true;
      for (int i = 0; i < sg.tiles; ++i, ++L) {
        const int s = L % NS;
        if (!(ok = warp_wait(smem_u32(&bar_full[s]), (L / NS) & 1, wc, 143))) break;
        const uint32_t sk = sbase + s * C::STAGE, sv = sk + C::TILE;
        const int key0 = (sg.kt0 + i) * kKeys + warp * 16;
        if (key0 < sg.keys) {
          // S = Q K^T for this warp's 16 keys: two n-tiles of 8, each in two sums.
          // A warp's latency through a stage is what small calls wait for, so the
          // fragments are fetched AHEAD steps before the product that takes them
          // (fetched one by one a stage took 1.3 us), V's first ones before the
          // softmax.  Q's come from shared memory for every stage: kept in
          // registers they would not fit beside O at two CTAs an SM.
          constexpr int AHEAD = 4;
          float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, sd[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
          const int krow = warp * 16 + (lane & 7) + ((lane >> 4) << 3), vrow = warp * 16 + (lane & 15);
          uint32_t fr[AHEAD][4], qf[AHEAD][4];
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {
            ldsm4(fr[k], swz(sk, C::SLAB, krow, 2 * k + ((lane >> 3) & 1)));
            ldsm4(qf[k], swz(sq, C::QSLAB, lane & 15, 2 * k + (lane >> 4)));
          }
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t(&b)[4] = fr[k % AHEAD];
            mma16816(k & 1 ? sd[0] : sc[0], qf[k % AHEAD], b[0], b[1]);
            mma16816(k & 1 ? sd[1] : sc[1], qf[k % AHEAD], b[2], b[3]);
            if (k + AHEAD < D / 16) {
              ldsm4(b, swz(sk, C::SLAB, krow, 2 * (k + AHEAD) + ((lane >> 3) & 1)));
              ldsm4(qf[k % AHEAD], swz(sq, C::QSLAB, lane & 15, 2 * (k + AHEAD) + (lane >> 4)));
            } else {
              ldsm4t(b, swz(sv, C::SLAB, vrow, 2 * ((k + AHEAD) % (D / 16)) + (lane >> 4)));
            }
          }
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] += sd[n][e];
          if (key0 + 16 > sg.ctx) {  // some key of the warp is a draft or behind the last
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // what the lane's row sees: up to its last key (chains), or the draft bits
              const int row = (lane >> 2) + 8 * h, j = sg.tok + (row < rows ? row / a.rep : 0);
              const int last_key = min(sg.ctx + j, sg.keys - 1);
              const unsigned long long see = a.mask != nullptr ? visible_drafts(a, sg, sg.row0 + j) : 0ull;
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int key = key0 + n * 8 + (lane & 3) * 2 + e, d = key - sg.ctx;
                  const bool vis = a.mask == nullptr ? key <= last_key : d < 0 || (d < 64 && (see >> (d & 63) & 1));
                  if (!vis) sc[n][2 * h + e] = neg_inf();
                }
            }
          }
          uint32_t pf[4];
          float alpha[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mx = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[h], mx * sl2);
            alpha[h] = ex2_approx(m[h] - mn);
            m[h] = mn;
            const float p0 = ex2_approx(fmaf(sc[0][2 * h], sl2, -mn)), p1 = ex2_approx(fmaf(sc[0][2 * h + 1], sl2, -mn));
            const float p2 = ex2_approx(fmaf(sc[1][2 * h], sl2, -mn)), p3 = ex2_approx(fmaf(sc[1][2 * h + 1], sl2, -mn));
            l[h] = l[h] * alpha[h] + ((p0 + p1) + (p2 + p3));
            pf[h] = pack_bf16x2(p0, p1);
            pf[h + 2] = pack_bf16x2(p2, p3);
          }
          if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
              o[d][0] *= alpha[0];
              o[d][1] *= alpha[0];
              o[d][2] *= alpha[1];
              o[d][3] *= alpha[1];
            }
          }
          // V's rows behind the last key: this lane's fragments hold keys key0 + (lane & 3) 2 (+1) (+8)
          uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
          const bool ragged = key0 + 16 > sg.keys;
          if (ragged) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int key = key0 + (lane & 3) * 2 + 8 * x;
              keep[x] = (key < sg.keys ? 0xffffu : 0u) | (key + 1 < sg.keys ? 0xffff0000u : 0u);
            }
          }
          // A product adds 0 V for the keys a row does not see, which is not 0
          // where V is infinite or NaN: drafts are looked through for such
          // values, and added without the matrix units where there are any.
          bool odd = false;
          if (key0 + 16 > sg.ctx && (a.mask != nullptr || sg.keys - sg.ctx > 1)) {
            for (int e = lane; e < 16 * (D / 8); e += 32) {
              const int r = e / (D / 8);
              if (key0 + r < sg.keys) odd |= nonfinite8(lds_u4(swz(sv, C::SLAB, warp * 16 + r, e % (D / 8))));
            }
            odd = __any_sync(0xffffffffu, odd);
          }
          if (odd) {
            for (int key = 0; key < 16 && key0 + key < sg.keys; ++key) {
              float p[2];
              bool seen[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t w = __shfl_sync(0xffffffffu, key < 8 ? pf[h] : pf[h + 2], (lane & ~3) | ((key & 7) >> 1));
                p[h] = __uint_as_float(key & 1 ? w & 0xffff0000u : w << 16);
                const int row = (lane >> 2) + 8 * h, j = sg.tok + (row < rows ? row / a.rep : 0), d = key0 + key - sg.ctx;
                seen[h] = a.mask == nullptr ? d <= j : d < 0 || (d < 64 && (visible_drafts(a, sg, sg.row0 + j) >> d & 1));
              }
#pragma unroll
              for (int d = 0; d < D / 8; ++d) {
                uint32_t w;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(swz(sv, C::SLAB, warp * 16 + key, d) + (lane & 3) * 4));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  if (!seen[h]) continue;
                  const float v0 = __uint_as_float(w << 16), v1 = __uint_as_float(w & 0xffff0000u);
                  // (a weight that underflowed is not 0: such a value is still itself)
                  o[d][2 * h] = p[h] == 0.f && !isfinite(v0) ? o[d][2 * h] + v0 : fmaf(p[h], v0, o[d][2 * h]);
                  o[d][2 * h + 1] = p[h] == 0.f && !isfinite(v1) ? o[d][2 * h + 1] + v1 : fmaf(p[h], v1, o[d][2 * h + 1]);
                }
              }
            }
          } else {
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              uint32_t(&b)[4] = fr[d % AHEAD];
              if (ragged) {
                b[0] &= keep[0];
                b[1] &= keep[1];
                b[2] &= keep[0];
                b[3] &= keep[1];
              }
              mma16816(o[2 * d], pf, b[0], b[1]);
              mma16816(o[2 * d + 1], pf, b[2], b[3]);
              if (d + AHEAD < D / 16) ldsm4t(b, swz(sv, C::SLAB, vrow, 2 * (d + AHEAD) + (lane >> 4)));
            }
          }
        }
        __syncwarp();
        if (i + 1 < sg.tiles && lane == 0) mbar_arrive(smem_u32(&bar_empty[s]));  // the last stage serves the join first
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_qempty[qs]));
      // ---- join the warps.  Each leaves its sums in the last stage, over the K and
      // V rows of its own 16 keys (which only it reads): 32 columns a slab, the
      // 16-byte chunks turned by the row as TMA does.  After one meeting all
      // threads join the four warps' sums, 4 columns of a row each.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      }
      float2(&ml)[kWarps][kRows] = stats[nj & 1];  // (segments without a stage do not meet)
      const uint32_t st = sbase + ((L + NS - 1) % NS) * C::STAGE;
      auto slab = [&](int p, int w) { return st + (p < D / 64 ? 0 : C::TILE) + p % (D / 64) * C::SLAB + w * 2048; };
      if (sg.tiles > 0) {
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = (lane >> 2) + 8 * h;
          if (8 * h >= rows) continue;
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            const uint32_t at = slab(d >> 2, warp) + row * 128 + ((((d & 3) * 2 + ((lane & 3) >> 1)) ^ (row & 7)) << 4) + (lane & 1) * 8;
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(o[d][2 * h]), "f"(o[d][2 * h + 1]) : "memory");
          }
          if ((lane & 3) == 0) ml[warp][row] = make_float2(m[h], l[h]);
        }
        if (!meet()) break;
      }
      // ---- out: o and lse, or this CTA's part (slot 0: the item began before, 1: it begins here)
      float* part = Part<kRows, D>::at(a, blockIdx.x, sg.first);
      for (int e = tid; e < rows * (D / 4); e += kWarps * 32) {
        const int row = e / (D / 4), c = e % (D / 4);  // columns 4 c .. 4 c + 3
        float mm = kFloor, ll = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (sg.tiles > 0) {
#pragma unroll
          for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[w][row].x);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 x = ml[w][row];
            if (x.y == 0.f) continue;  // no key of this warp's is seen
            const float f = ex2_approx(x.x - mm);
            const float4 v = lds_f4(slab(c >> 3, w) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
            ll = fmaf(f, x.y, ll);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
          }
        }
        if constexpr (CL) {  // to the cluster: over the query slots that a single segment leaves free
          st_shared_v4(sbase + C::OFF_Q + C::QSLOT + row * (D * 4) + c * 16, __float_as_uint(acc.x), __float_as_uint(acc.y),
                       __float_as_uint(acc.z), __float_as_uint(acc.w));
          if (c == 0) part_stats[row] = make_float2(mm, ll);
        } else if (sg.whole) {
          const int jt = row / a.rep, head = sg.kvh * a.rep + row - jt * a.rep, tk = sg.row0 + sg.tok + jt;
          const float inv = ll == 0.f ? 0.f : 1.f / ll;
          if (!row_in(a, tk, head, 745)) continue;
          *reinterpret_cast<uint2*>(a.o + (static_cast<size_t>(tk) * a.H + head) * D + 4 * c) =
              make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
          if (c == 0) a.lse[static_cast<size_t>(head) * a.T + tk] = lse_of(mm, ll);
        } else {
          *reinterpret_cast<float4*>(part + row * D + 4 * c) = acc;
          if (c == 0) {
            part[kRows * D + row] = mm;
            part[kRows * (D + 1) + row] = ll;
          }
        }
      }
      if (sg.tiles > 0) {
        fence_proxy_async_smem();  // these accesses before the TMA that refills the stage
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_empty[(L + NS - 1) % NS]));
      }
      if (!CL && tid == 0 && sg.first && !sg.whole && in_bounds(a.status, sg.last_cta, gridDim.x, 747))
        // join work: the parts lie in CTAs blockIdx.x .. last_cta
        a.desc[blockIdx.x] = join_work(sg);
    }
  }
  if constexpr (CL) {
    // A CTA that gave up a wait comes here too: the reads stay in shared memory
    // of CTAs that have not ended, whatever it holds.
    static_assert(kRows * D * 4 <= 2 * C::QSLOT, "the part fits the free query slots");
    cluster_meet();
    if (warp == kWarps && lane == 0 && *wc.abort) {
      drain_ring(smem_u32(bar_qfull), NQ, 1);
      drain_ring(smem_u32(bar_full), NS, only.tiles);
    }
    const int rows = only.ntok * a.rep, parts = cluster_size();
    if (warp < kWarps)
      for (int e = cluster_rank() * (kWarps * 32) + tid; e < rows * (D / 4); e += parts * (kWarps * 32)) {
        const int row = e / (D / 4), c = e % (D / 4);
        const uint32_t sums_at = sbase + C::OFF_Q + C::QSLOT + row * (D * 4) + c * 16, stat_at = smem_u32(&part_stats[row]);
        float mm = kFloor, ll = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int p = 0; p < parts; ++p) {
          const float2 x = ld_peer_f2(peer_addr(stat_at, p));
          const float4 v = ld_peer_f4(peer_addr(sums_at, p));
          if (x.y == 0.f) continue;  // no key of this part is seen
          const float mn = fmaxf(mm, x.x), fo = ex2_approx(mm - mn), f = ex2_approx(x.x - mn);
          mm = mn;
          ll = fo * ll + f * x.y;
          acc.x = fmaf(fo, acc.x, f * v.x);
          acc.y = fmaf(fo, acc.y, f * v.y);
          acc.z = fmaf(fo, acc.z, f * v.z);
          acc.w = fmaf(fo, acc.w, f * v.w);
        }
        const int jt = row / a.rep, head = only.kvh * a.rep + row - jt * a.rep, tk = only.row0 + only.tok + jt;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        if (!row_in(a, tk, head, 746)) continue;
        *reinterpret_cast<uint2*>(a.o + (static_cast<size_t>(tk) * a.H + head) * D + 4 * c) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (c == 0) a.lse[static_cast<size_t>(head) * a.T + tk] = lse_of(mm, ll);
      }
    cluster_meet();  // no CTA leaves while its memory is read
  }
}

template <int D>
cudaError_t dec_launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CacheAttnArgs& a,
                       int grid, int cluster, cudaStream_t stream) {
  auto* const kernel = cluster > 0 ? s2_cache_dec_kernel<D, true> : s2_cache_dec_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, DecCfg<D>::SMEM);
  if (e == cudaSuccess && cluster > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kDecThreads);
  cfg.dynamicSmemBytes = DecCfg<D>::SMEM;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  prof_before(stream, kKernelCacheAttn);
  e = cudaLaunchKernelEx(&cfg, kernel, tq, tk, tv, a);
  prof_after(stream);
  if (e != cudaSuccess || cluster > 0) return e;
  return launch_join<kRows, kRows, D, 4, 1>(a, grid, stream);
}

}  // namespace

cudaError_t launch_cache_dec(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CacheAttnArgs& a,
                             int D, int grid, int cluster, cudaStream_t stream) {
  return D == 64 ? dec_launch<64>(tq, tk, tv, a, grid, cluster, stream)
                 : dec_launch<128>(tq, tk, tv, a, grid, cluster, stream);
}

}  // namespace s2
