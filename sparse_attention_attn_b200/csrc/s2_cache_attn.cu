// Attention of new tokens over a paged cache: one token, a chain or a tree of
// drafts for each request of a ragged batch.
//
//   o = softmax(q K^T / sqrt(D), masked) V,  lse = log sum exp (natural log)
//
// Token j of request i (rows cu[i] .. cu[i+1]) sees every key before ctx_i and,
// of the request's own new keys, those its mask names (bit j' = draft j'), or
// without masks the drafts up to itself.  Key p of request i is row p % bs of
// cache block block_table[i][p / bs].
//
// Rows.  The rep = H/Hkv query heads that share a kv head form one tile with
// the request's tokens: row = j * rep + (head in its group), 16 rows a tile.
//
// Split.  A unit is one tile of 64 keys of one (request, kv head, row tile);
// all units of a batch are numbered in that order and dealt to the CTAs in
// equal contiguous runs, so a batch of very different lengths, or one long
// request, loads every SM alike.  A run that covers only a part of an item's
// keys leaves its unnormalised sums, row maxima and row sums in the workspace,
// and a second kernel joins the parts in order: a fixed split, so the same
// call gives the same bits.
//
// Within a CTA each of four warps takes 16 of a tile's 64 keys through
// mma.sync with its own running maximum and sum (fp32), joined at the item's
// end; P is rounded to bf16 for the product with V, as in the training
// kernels, its row sums are taken before the rounding.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "s2_common.cuh"
#include "s2_ptx.cuh"

namespace s2 {

namespace {

constexpr int kRows = kCacheRows;  // rows of a tile
constexpr int kKeys = 64;          // keys of a tile
constexpr int kWarps = 4;
constexpr int kStages = 3;

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
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// 16 bytes global -> shared, or 16 zero bytes when !live (nothing is read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The lengths of request i, and its units.
struct Req {
  int ctx, n, row0;  // cached tokens, new tokens, first row of q
  int keys;          // ctx + n
  int kt, rt;        // key tiles, row tiles
  long long units;   // Hkv * rt * kt
};
__device__ __forceinline__ Req request(const CacheAttnArgs& a, int i) {
  Req r;
  r.row0 = min(max(a.cu_seqlens[i], 0), a.T);
  const int end = min(max(a.cu_seqlens[i + 1], r.row0), a.T);
  r.n = end - r.row0;
  const long long most = static_cast<long long>(a.max_blocks) << a.bs_log2;  // places the table has
  r.ctx = static_cast<int>(min(static_cast<long long>(max(a.ctx_lens[i], 0)), most));
  r.keys = static_cast<int>(min(static_cast<long long>(r.ctx) + r.n, most));
  r.kt = (r.keys + kKeys - 1) / kKeys;
  if (r.kt == 0) r.kt = 1;  // rows without a key still get their zeros
  r.rt = static_cast<int>((static_cast<long long>(r.n) * a.rep + kRows - 1) / kRows);
  r.units = static_cast<long long>(a.Hkv) * r.rt * r.kt;
  return r;
}

// Sum of v over the block's threads (kWarps * 32); every thread gets it.
__device__ __forceinline__ long long block_sum(long long v, long long* buf) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += buf[w];
  return v;
}

template <int D>
struct Smem {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kTileBytes = kKeys * kRowBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;  // K and V
  static constexpr int kBytes = kStages * kStageBytes + 1024;
  static_assert(kStages * kStageBytes >= kWarps * kRows * (D + 4) * 4 + 2 * kWarps * kRows * 4, "join buffers");
};

// Byte offset of 16-byte chunk c of row r: the chunk index is turned by the
// row so that the 8 rows of an ldmatrix (and of a cp.async warp) hit 8
// different bank groups.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return static_cast<uint32_t>(r) * (D * 2) + static_cast<uint32_t>((c ^ (r & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) s2_cache_attn_kernel(CacheAttnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t sbase = smem_u32(smem);
  __shared__ long long sums[kWarps];
  __shared__ long long scan[kWarps * 32 + 1];
  __shared__ int found[2];
  __shared__ long long found_before;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // ---- the run of units of this CTA
  long long total = 0;
  for (int base = 0; base < a.R; base += kWarps * 32) {
    const int i = base + tid;
    total += block_sum(i < a.R ? request(a, i).units : 0, sums);
  }
  const long long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(kCacheMinUnits));
  const long long u0 = per * blockIdx.x, u1 = min(u0 + per, total);
  int4* desc = a.desc + blockIdx.x;
  if (tid == 0) *desc = make_int4(-1, 0, 0, 0);
  if (u0 >= u1) return;
  // ---- the request of unit u0
  long long before = 0;
  for (int base = 0; base < a.R; base += kWarps * 32) {
    const int i = base + tid;
    const long long mine = i < a.R ? request(a, i).units : 0;
    const long long all = block_sum(mine, sums);
    if (u0 < before + all) {  // in this chunk (uniform)
      scan[tid] = mine;
      __syncthreads();
      if (tid == 0) {
        long long x = before;
        int k = 0;
        while (x + scan[k] <= u0) x += scan[k++];
        found[0] = base + k;
        found_before = x;
      }
      __syncthreads();
      break;
    }
    before += all;
  }
  int ri = found[0];
  long long rbase = found_before;
  const float sl2 = a.scale_log2;
  for (long long u = u0; u < u1;) {
    Req r = request(a, ri);
    if (u >= rbase + r.units) {
      rbase += r.units;
      ++ri;
      continue;
    }
    const long long in = u - rbase;
    const int kt0 = static_cast<int>(in % r.kt);
    const long long item = in / r.kt;  // kvh * rt + row tile
    const int rt = static_cast<int>(item % r.rt), kvh = static_cast<int>(item / r.rt);
    const int kt1 = static_cast<int>(min(static_cast<long long>(r.kt), kt0 + (u1 - u)));
    u += kt1 - kt0;
    const int* table = a.block_tables + static_cast<size_t>(ri) * a.max_blocks;
    // the last key any row of the tile sees (chain: its last token's own)
    const int rows = min(kRows, r.n * a.rep - rt * kRows);
    const int j_last = (rt * kRows + rows - 1) / a.rep;
    const int reach = a.mask != nullptr ? r.keys : min(r.ctx + min(j_last + 1, r.keys - r.ctx), r.keys);
    const int t_end = min(kt1, (reach + kKeys - 1) / kKeys);
    // ---- Q fragments: rows lane/4 and lane/4 + 8
    uint32_t qf[D / 16][4];
    int tok[2], jrow[2];
    unsigned long long see[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = rt * kRows + (lane >> 2) + 8 * h;
      const bool live = row < r.n * a.rep;
      const int j = live ? row / a.rep : 0, g = live ? row - j * a.rep : 0;
      tok[h] = r.row0 + j;
      jrow[h] = j;
      see[h] = a.mask != nullptr ? a.mask[tok[h]] : 0ull;
      const __nv_bfloat16* src = a.q + (static_cast<size_t>(tok[h]) * a.H + kvh * a.rep + g) * D + (lane & 3) * 2;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][h] = live ? *reinterpret_cast<const uint32_t*>(src + k * 16) : 0u;
        qf[k][h + 2] = live ? *reinterpret_cast<const uint32_t*>(src + k * 16 + 8) : 0u;
      }
    }
    auto load_tile = [&](int t, int stage) {
      const uint32_t sk = sbase + stage * Smem<D>::kStageBytes, sv = sk + Smem<D>::kTileBytes;
      constexpr int CPR = D / 8;  // 16-byte chunks of a row
#pragma unroll
      for (int x = 0; x < kKeys * CPR / (kWarps * 32); ++x) {
        const int e = x * (kWarps * 32) + tid, row = e / CPR, c = e % CPR;
        const int key = t * kKeys + row;
        bool live = key < r.keys;
        const int blk = live ? table[key >> a.bs_log2] : 0;
        live = live && data_in_range(a.status, blk, a.num_blocks, 711);
        const size_t place = (static_cast<size_t>(blk) << a.bs_log2) + (key & ((1 << a.bs_log2) - 1));
        const size_t off = live ? (place * a.Hkv + kvh) * D + c * 8 : 0;
        cp16(sk + swz<D>(row, c), a.k_cache + off, live);
        cp16(sv + swz<D>(row, c), a.v_cache + off, live);
      }
    };
    float o[D / 8][4];
#pragma unroll
    for (int d = 0; d < D / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      if (kt0 + s < t_end) load_tile(kt0 + s, s);
      cp_commit();
    }
    for (int t = kt0; t < t_end; ++t) {
      cp_wait<kStages - 2>();
      __syncthreads();
      const int nx = t + kStages - 1;
      if (nx < t_end) load_tile(nx, (nx - kt0) % kStages);
      cp_commit();
      const uint32_t sk = sbase + ((t - kt0) % kStages) * Smem<D>::kStageBytes, sv = sk + Smem<D>::kTileBytes;
      // S = Q K^T for this warp's 16 keys: two n-tiles of 8
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const int krow = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldsm4(b, sk + swz<D>(krow, 2 * k + ((lane >> 3) & 1)));
        mma16816(s[0], qf[k], b[0], b[1]);
        mma16816(s[1], qf[k], b[2], b[3]);
      }
      const int key0 = t * kKeys + warp * 16;
      const bool edge = key0 + 16 > r.ctx;  // some key of the warp is a draft or behind the last
      if (edge) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + n * 8 + (lane & 3) * 2 + (e & 1), h = e >> 1, d = key - r.ctx;
            const bool vis = d < 0 || (key < r.keys && (a.mask != nullptr ? (d < 64 && (see[h] >> (d & 63) & 1)) : d <= jrow[h]));
            if (!vis) s[n][e] = neg_inf();
          }
      }
      uint32_t pf[4];
      float alpha[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[h], mx * sl2);
        const float base = mn == neg_inf() ? 0.f : mn;
        alpha[h] = ex2_approx(m[h] - base);
        m[h] = mn;
        const float p0 = ex2_approx(fmaf(s[0][2 * h], sl2, -base)), p1 = ex2_approx(fmaf(s[0][2 * h + 1], sl2, -base));
        const float p2 = ex2_approx(fmaf(s[1][2 * h], sl2, -base)), p3 = ex2_approx(fmaf(s[1][2 * h + 1], sl2, -base));
        l[h] = l[h] * alpha[h] + (p0 + p1) + (p2 + p3);
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
      const int vrow = warp * 16 + (lane & 15);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t b[4];
        ldsm4t(b, sv + swz<D>(vrow, 2 * d + (lane >> 4)));
        mma16816(o[2 * d], pf, b[0], b[1]);
        mma16816(o[2 * d + 1], pf, b[2], b[3]);
      }
    }
    cp_wait<0>();
    // ---- join the warps
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    __syncthreads();  // the stages are free
    float* jo = reinterpret_cast<float*>(smem);          // [warp][row][D + 4]
    float* jm = jo + kWarps * kRows * (D + 4);           // [warp][row]
    float* jl = jm + kWarps * kRows;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = (lane >> 2) + 8 * h;
      float* dst = jo + (warp * kRows + row) * (D + 4) + (lane & 3) * 2;
#pragma unroll
      for (int d = 0; d < D / 8; ++d) *reinterpret_cast<float2*>(dst + d * 8) = make_float2(o[d][2 * h], o[d][2 * h + 1]);
      if ((lane & 3) == 0) {
        jm[warp * kRows + row] = m[h];
        jl[warp * kRows + row] = l[h];
      }
    }
    __syncthreads();
    const bool whole = kt0 == 0 && kt1 == r.kt;
    const int slot = 2 * blockIdx.x + (kt0 == 0 ? 1 : 0);  // 1: an item begins here, 0: it began before
    float* part = a.partial + static_cast<size_t>(slot) * kRows * (D + 2);
    for (int e = tid; e < kRows * (D / 4); e += kWarps * 32) {
      const int row = e / (D / 4), c = (e % (D / 4)) * 4;
      if (row >= rows) continue;
      float mm = neg_inf();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, jm[w * kRows + row]);
      const float base = mm == neg_inf() ? 0.f : mm;
      float ll = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(jm[w * kRows + row] - base);
        const float4 v = *reinterpret_cast<const float4*>(jo + (w * kRows + row) * (D + 4) + c);
        ll = fmaf(f, jl[w * kRows + row], ll);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      if (whole) {
        const int gr = rt * kRows + row, j = gr / a.rep, h = kvh * a.rep + gr - j * a.rep, tk = r.row0 + j;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        *reinterpret_cast<uint2*>(a.o + (static_cast<size_t>(tk) * a.H + h) * D + c) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (c == 0) a.lse[static_cast<size_t>(h) * a.T + tk] = ll == 0.f ? neg_inf() : (mm + log2f(ll)) * 0.69314718055994531f;
      } else {
        *reinterpret_cast<float4*>(part + row * D + c) = acc;
        if (c == 0) {
          part[kRows * D + row] = mm;
          part[kRows * D + kRows + row] = ll;
        }
      }
    }
    if (!whole && kt0 == 0 && tid == 0) {  // this CTA's join work: the item's parts lie in CTAs blockIdx.x .. last
      const long long item_end = rbase + (item + 1) * r.kt;
      *desc = make_int4(ri, static_cast<int>(item / r.rt), rt, static_cast<int>((item_end - 1) / per));
    }
    __syncthreads();  // the join buffers become stages again
  }
}

// Joins the parts of the items that more than one CTA worked on: block b the
// item that begins in CTA b and runs on.  Warp w takes rows w, w + 8, ...
template <int D>
__global__ void __launch_bounds__(256) s2_cache_merge_kernel(CacheAttnArgs a) {
  const int4 d = a.desc[blockIdx.x];
  if (d.x < 0) return;
  const Req r = request(a, d.x);
  const int kvh = d.y, rt = d.z, last = d.w, first = blockIdx.x;
  const int rows = min(kRows, r.n * a.rep - rt * kRows);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int PER = D / 32;
  constexpr size_t kSlot = kRows * (D + 2);
  for (int row = warp; row < rows; row += 8) {
    float mm = neg_inf();
    for (int b = first; b <= last; ++b) mm = fmaxf(mm, a.partial[(2 * b + (b == first)) * kSlot + kRows * D + row]);
    const float base = mm == neg_inf() ? 0.f : mm;
    float ll = 0.f, acc[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[k] = 0.f;
    for (int b = first; b <= last; ++b) {
      const float* part = a.partial + (2 * b + (b == first)) * kSlot;
      const float f = ex2_approx(part[kRows * D + row] - base);
      ll = fmaf(f, part[kRows * D + kRows + row], ll);
#pragma unroll
      for (int k = 0; k < PER; ++k) acc[k] = fmaf(f, part[row * D + lane * PER + k], acc[k]);
    }
    const int gr = rt * kRows + row, j = gr / a.rep, h = kvh * a.rep + gr - j * a.rep, tk = r.row0 + j;
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.o + (static_cast<size_t>(tk) * a.H + h) * D + lane * PER);
#pragma unroll
    for (int k = 0; k < PER / 2; ++k) out[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    if (lane == 0) a.lse[static_cast<size_t>(h) * a.T + tk] = ll == 0.f ? neg_inf() : (mm + log2f(ll)) * 0.69314718055994531f;
  }
}

template <int D>
cudaError_t attn_launch(const CacheAttnArgs& a, int grid, cudaStream_t stream) {
  const cudaError_t ea =
      cudaFuncSetAttribute(s2_cache_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
  if (ea != cudaSuccess) return ea;
  prof_before(stream, kKernelCacheAttn);
  s2_cache_attn_kernel<D><<<grid, kWarps * 32, Smem<D>::kBytes, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  prof_after(stream);
  if (e != cudaSuccess) return e;
  prof_before(stream, kKernelCacheMerge);
  s2_cache_merge_kernel<D><<<grid, 256, 0, stream>>>(a);
  e = cudaGetLastError();
  prof_after(stream);
  return e;
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int D, int grid, cudaStream_t stream) {
  return D == 64 ? attn_launch<64>(a, grid, stream) : attn_launch<128>(a, grid, stream);
}

}  // namespace s2
