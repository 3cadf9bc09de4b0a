// Root-mean-square norm of every query and key head with a learned weight,
// and the rotation by position, in one pass; its backward; and the serving
// form, which takes the new tokens of a ragged batch at any positions and puts
// the rotated keys and the values into their slots of a paged cache.
//
// For a head row x of D values at position t:
//   r = 1 / sqrt(mean(x^2) + eps),  u = r x w,  y = R(a_t) u
// with R the rotation of the pairs (i, i + D/2) by the table's (cos, sin).
// Backward, from dy:  du = R(-a_t) dy,  dw = sum over rows of du r x,
//   g = du w,  dx = r (g - r^2 x mean(g x)).
// The row statistic is recomputed from x, so the forward stores nothing
// besides y.  All arithmetic is fp32; y, dx and (for bf16 weights) dw are
// rounded once.
//
// Every kernel is bound by HBM bytes at size (4 bytes a value forward, 6
// backward).  D/16 lanes hold one row -- 8 values of each half per lane, so a
// rotation pair never leaves its thread -- and reduce the row's sum by
// shuffles; a thread walks a group of heads of one token with the token's 8
// (cos, sin) pairs in registers.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "s2_common.cuh"
#include "s2_ptx.cuh"

namespace s2 {

namespace {

// 8 weights of one half at w + off, as fp32.
__device__ __forceinline__ void load_w8(const float* w, int off, float (&o)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(w + off), b = *reinterpret_cast<const float4*>(w + off + 4);
  o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&o)[8]) {
  const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&p[j]));
    o[2 * j] = f.x;
    o[2 * j + 1] = f.y;
  }
}
__device__ __forceinline__ void load_w8(const __nv_bfloat16* w, int off, float (&o)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(w + off), o);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void load_turn(const float2* table, size_t off, float (&c)[8], float (&s)[8]) {
  const float4* tp = reinterpret_cast<const float4*>(table + off);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = tp[j];
    c[2 * j] = v.x, s[2 * j] = v.y, c[2 * j + 1] = v.z, s[2 * j + 1] = v.w;
  }
}

// The backward's octets as 4 packed pairs: its arithmetic runs on pairs
// (fma.rn.f32x2), which halves its instructions (297 us at 32768 tokens x 72
// heads of 128, 318 on single floats, which filled half of the issue slots).
// The forward, with less arithmetic a byte, is faster on single floats (58 us at
// 16384 x 40 heads, 61 on pairs; the appended prompts of 16K tokens 130 and 138).
struct Oct {
  uint64_t v[4];
};
__device__ __forceinline__ Oct unpack_oct(const uint4& u) {
  const uint32_t p[4] = {u.x, u.y, u.z, u.w};
  Oct o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o.v[j] = f2_pack(__uint_as_float(p[j] << 16), __uint_as_float(p[j] & 0xffff0000u));
  return o;
}
__device__ __forceinline__ uint4 pack8(const Oct& f) {
  return make_uint4(f2_to_bf16x2(f.v[0]), f2_to_bf16x2(f.v[1]), f2_to_bf16x2(f.v[2]), f2_to_bf16x2(f.v[3]));
}
// 8 weights of one half at w + off, as fp32.
__device__ __forceinline__ Oct load_oct(const float* w, int off) {
  const float4 a = *reinterpret_cast<const float4*>(w + off), b = *reinterpret_cast<const float4*>(w + off + 4);
  return {{f2_pack(a.x, a.y), f2_pack(a.z, a.w), f2_pack(b.x, b.y), f2_pack(b.z, b.w)}};
}
__device__ __forceinline__ Oct load_oct(const __nv_bfloat16* w, int off) {
  return unpack_oct(*reinterpret_cast<const uint4*>(w + off));
}
// cos, sin and -sin of 8 pairs
__device__ __forceinline__ void load_turn_oct(const float2* table, size_t off, Oct& c, Oct& s, Oct& ns) {
  const float4* tp = reinterpret_cast<const float4*>(table + off);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = tp[j];
    c.v[j] = f2_pack(v.x, v.z);
    s.v[j] = f2_pack(v.y, v.w);
    ns.v[j] = f2_pack(-v.y, -v.w);
  }
}
__device__ __forceinline__ float f2_sum(uint64_t v) { return f2_lo(v) + f2_hi(v); }

// Sum over the CH (4 or 8) lanes of a row; all 32 lanes of the warp take part.
template <int CH>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = CH / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// 1 / sqrt(mean(x^2) + eps) of a row, this lane holding x1 and x2
template <int D>
__device__ __forceinline__ float row_rms(const Oct& x1, const Oct& x2, float eps) {
  uint64_t sa = f2_mul(x1.v[0], x1.v[0]), sb = f2_mul(x2.v[0], x2.v[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) {
    sa = f2_fma(x1.v[j], x1.v[j], sa);
    sb = f2_fma(x2.v[j], x2.v[j], sb);
  }
  return rsqrtf(row_sum<D / 16>(f2_sum(f2_add(sa, sb))) * (1.f / D) + eps);
}

// y = R(a) (r x w) of one lane's two octets; NORM false: r x w = x.
template <int D, bool NORM>
__device__ __forceinline__ void norm_rope_row(const uint4& u1, const uint4& u2, const float (&w1)[8],
                                              const float (&w2)[8], const float (&c)[8], const float (&s)[8],
                                              float eps, uint4& o1, uint4& o2) {
  float x1[8], x2[8], y1[8], y2[8];
  unpack8(u1, x1);
  unpack8(u2, x2);
  if (NORM) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x1[j], x1[j], fmaf(x2[j], x2[j], ss));
    const float r = rsqrtf(row_sum<D / 16>(ss) * (1.f / D) + eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x1[j] *= r * w1[j];
      x2[j] *= r * w2[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y1[j] = fmaf(x1[j], c[j], -x2[j] * s[j]);
    y2[j] = fmaf(x1[j], s[j], x2[j] * c[j]);
  }
  o1 = pack8(y1);
  o2 = pack8(y2);
}

// Forward.  A unit is a group of HG heads of one token (the query groups, then
// the key groups); D/16 lanes take one unit.  Loops run on whole warps so that
// the shuffles always have all lanes.
template <int D, typename W, int HG>
__global__ void __launch_bounds__(256) s2_qknorm_fwd_kernel(QkNormArgs a) {
  constexpr int CH = D / 16;
  const int gq = (a.H + HG - 1) / HG, gk = (a.Hkv + HG - 1) / HG, G = gq + gk;
  const long long n = static_cast<long long>(a.tokens) * G * CH;
  for (long long e0 = blockIdx.x * 256LL + (threadIdx.x & ~31u); e0 < n; e0 += gridDim.x * 256LL) {
    const long long e = e0 + (threadIdx.x & 31u);
    bool live = e < n;
    const int ch = static_cast<int>(e % CH);
    const uint32_t unit = live ? static_cast<uint32_t>(e / CH) : 0u;  // < 2^31 (checked by the host)
    const int tok = unit / G, gi = unit - tok * G;
    const bool is_q = gi < gq;
    const int h0 = (is_q ? gi : gi - gq) * HG, heads = is_q ? a.H : a.Hkv;
    const __nv_bfloat16* src = (is_q ? a.q : a.k) + (static_cast<size_t>(tok) * heads + h0) * D + ch * 8;
    __nv_bfloat16* dst = (is_q ? a.yq : a.yk) + (static_cast<size_t>(tok) * heads + h0) * D + ch * 8;
    live = live && in_bounds(a.status, tok, a.tokens, 720) && in_bounds(a.status, h0, heads, 721);
    uint4 u1[HG], u2[HG];
#pragma unroll
    for (int k = 0; k < HG; ++k) {
      u1[k] = u2[k] = make_uint4(0, 0, 0, 0);
      if (live && h0 + k < heads) {
        u1[k] = *reinterpret_cast<const uint4*>(src + k * D);
        u2[k] = *reinterpret_cast<const uint4*>(src + k * D + D / 2);
      }
    }
    float c[8], s[8], w1[8], w2[8];
    load_turn(a.table, static_cast<size_t>(tok % a.N) * (D / 2) + ch * 8, c, s);
    const W* w = static_cast<const W*>(is_q ? a.wq : a.wk);
    load_w8(w, ch * 8, w1);
    load_w8(w, ch * 8 + D / 2, w2);
#pragma unroll
    for (int k = 0; k < HG; ++k) {
      uint4 o1, o2;
      norm_rope_row<D, true>(u1[k], u2[k], w1, w2, c, s, a.eps, o1, o2);
      if (live && h0 + k < heads) {
        *reinterpret_cast<uint4*>(dst + k * D) = o1;
        *reinterpret_cast<uint4*>(dst + k * D + D / 2) = o2;
      }
    }
  }
}

// Backward.  The same units; the first blocks take the query rows and the others
// the key rows, HG heads of a token at a time.  A thread keeps the sums of du r x
// of its 16 columns in registers, and the block leaves a partial row in the
// workspace.  Two blocks an SM (128 registers a thread) with two heads a thread
// keep 64 KB of loads in flight there; at 32768 tokens x 72 heads of 128: 297-308
// us of 280 at the measured copy bandwidth.  Measured on the way: 409 us with one
// block an SM, 342 with four heads a thread, 580 with one head and three blocks
// (spills), 382 with chunks bulk-copied through a shared-memory ring, whose extra
// instructions cost more than the loads in flight gave.
template <int D, typename W, int HG>
__global__ void __launch_bounds__(256, 2) s2_qknorm_bwd_kernel(QkNormArgs a) {
  constexpr int CH = D / 16;
  __shared__ float red[8][D];
  launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ch = lane % CH;
  const bool which = static_cast<int>(blockIdx.x) >= a.blocks_q;  // key rows
  const int block = which ? blockIdx.x - a.blocks_q : blockIdx.x, grid = which ? a.blocks - a.blocks_q : a.blocks_q;
  const int heads = which ? a.Hkv : a.H;
  const __nv_bfloat16* x = which ? a.k : a.q;
  const __nv_bfloat16* dy = which ? a.gk : a.gq;
  __nv_bfloat16* dx = which ? a.yk : a.yq;
  const W* w = static_cast<const W*>(which ? a.wk : a.wq);
  const Oct w1 = load_oct(w, ch * 8), w2 = load_oct(w, ch * 8 + D / 2);
  Oct acc1 = {{0ull, 0ull, 0ull, 0ull}}, acc2 = acc1;
  const int G = (heads + HG - 1) / HG;
  const long long n = static_cast<long long>(a.tokens) * G * CH;
  for (long long e0 = block * 256LL + (threadIdx.x & ~31u); e0 < n; e0 += grid * 256LL) {
    const long long e = e0 + lane;
    bool live = e < n;
    const uint32_t unit = live ? static_cast<uint32_t>(e / CH) : 0u;
    const int tok = unit / G, h0 = (unit - tok * G) * HG;
    live = live && in_bounds(a.status, tok, a.tokens, 722) && in_bounds(a.status, h0, heads, 723);
    const size_t off = (static_cast<size_t>(tok) * heads + h0) * D + ch * 8;
    uint4 u1[HG], u2[HG], d1[HG], d2[HG];
#pragma unroll
    for (int k = 0; k < HG; ++k) {
      u1[k] = u2[k] = d1[k] = d2[k] = make_uint4(0, 0, 0, 0);
      if (live && h0 + k < heads) {
        u1[k] = *reinterpret_cast<const uint4*>(x + off + k * D);
        u2[k] = *reinterpret_cast<const uint4*>(x + off + k * D + D / 2);
        d1[k] = *reinterpret_cast<const uint4*>(dy + off + k * D);
        d2[k] = *reinterpret_cast<const uint4*>(dy + off + k * D + D / 2);
      }
    }
    Oct c, s, ns;
    load_turn_oct(a.table, static_cast<size_t>(tok % a.N) * (D / 2) + ch * 8, c, s, ns);
#pragma unroll
    for (int k = 0; k < HG; ++k) {
      const Oct x1 = unpack_oct(u1[k]), x2 = unpack_oct(u2[k]);
      Oct g1 = unpack_oct(d1[k]), g2 = unpack_oct(d2[k]);
      const float r = row_rms<D>(x1, x2, a.eps);
      const uint64_t r2 = f2_pack(r, r);
      uint64_t sa = 0ull, sb = 0ull;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // du, then dw += du r x, g = du w, sum of g x
        const uint64_t du1 = f2_fma(g2.v[j], s.v[j], f2_mul(g1.v[j], c.v[j]));
        const uint64_t du2 = f2_fma(g1.v[j], ns.v[j], f2_mul(g2.v[j], c.v[j]));
        acc1.v[j] = f2_fma(du1, f2_mul(r2, x1.v[j]), acc1.v[j]);
        acc2.v[j] = f2_fma(du2, f2_mul(r2, x2.v[j]), acc2.v[j]);
        g1.v[j] = f2_mul(du1, w1.v[j]);
        g2.v[j] = f2_mul(du2, w2.v[j]);
        sa = f2_fma(g1.v[j], x1.v[j], sa);
        sb = f2_fma(g2.v[j], x2.v[j], sb);
      }
      const float nm = row_sum<CH>(f2_sum(f2_add(sa, sb))) * (-1.f / D) * r * r;
      const uint64_t nm2 = f2_pack(nm, nm);
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // dx = r (g - r^2 mean(g x) x)
        g1.v[j] = f2_mul(r2, f2_fma(x1.v[j], nm2, g1.v[j]));
        g2.v[j] = f2_mul(r2, f2_fma(x2.v[j], nm2, g2.v[j]));
      }
      if (live && h0 + k < heads) {
        *reinterpret_cast<uint4*>(dx + off + k * D) = pack8(g1);
        *reinterpret_cast<uint4*>(dx + off + k * D + D / 2) = pack8(g2);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // lanes of equal chunk, then the block's warps
#pragma unroll
    for (int m = CH; m < 32; m <<= 1) {
      acc1.v[j] = f2_add(acc1.v[j], __shfl_xor_sync(0xffffffffu, acc1.v[j], m));
      acc2.v[j] = f2_add(acc2.v[j], __shfl_xor_sync(0xffffffffu, acc2.v[j], m));
    }
  }
  if (lane < CH) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      red[warp][ch * 8 + 2 * j] = f2_lo(acc1.v[j]);
      red[warp][ch * 8 + 2 * j + 1] = f2_hi(acc1.v[j]);
      red[warp][ch * 8 + D / 2 + 2 * j] = f2_lo(acc2.v[j]);
      red[warp][ch * 8 + D / 2 + 2 * j + 1] = f2_hi(acc2.v[j]);
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[i][threadIdx.x];
    if (in_bounds(a.status, blockIdx.x, kQkNormMaxBlocks, 724))
      a.partial[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = t;
  }
}

// Sums the blocks' partial weight gradients (in fp64, in block order within
// each of the 32 strides, so a result does not depend on timing).
__device__ __forceinline__ void store_w(float* p, int i, double v) { p[i] = static_cast<float>(v); }
__device__ __forceinline__ void store_w(__nv_bfloat16* p, int i, double v) { p[i] = __double2bfloat16(v); }

template <int D, typename W>
__global__ void __launch_bounds__(1024) s2_qknorm_dw_kernel(QkNormArgs a) {
  __shared__ double red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool which = blockIdx.x >= D / 32;
  const int col = blockIdx.x % (D / 32) * 32 + lane;
  wait_for_primary();
  if (!in_bounds(a.status, a.blocks - 1, kQkNormMaxBlocks, 725)) return;
  double t = 0.0;
  for (int b = (which ? a.blocks_q : 0) + warp; b < (which ? a.blocks : a.blocks_q); b += 32)
    t += a.partial[static_cast<size_t>(b) * D + col];
  red[warp][lane] = t;
  __syncthreads();
  if (warp == 0) {
    t = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += red[i][lane];
    store_w(static_cast<W*>(which ? a.dwk : a.dwq), col, t);
  }
}

// Serving form.  Units of a token: its query groups, key groups and value
// groups.  A token whose slot is negative is padding: nothing of it is
// written.  Positions outside the table and slots outside the cache are
// recorded in the device status and the token is skipped.
template <int D, typename W, bool NORM, int HG>
__global__ void __launch_bounds__(256) s2_cache_append_kernel(CacheAppendArgs a) {
  constexpr int CH = D / 16;
  const int gq = (a.H + HG - 1) / HG, gk = (a.Hkv + HG - 1) / HG, G = gq + 2 * gk;
  const long long n = static_cast<long long>(a.T) * G * CH;
  for (long long e0 = blockIdx.x * 256LL + (threadIdx.x & ~31u); e0 < n; e0 += gridDim.x * 256LL) {
    const long long e = e0 + (threadIdx.x & 31u);
    bool live = e < n;
    const int ch = static_cast<int>(e % CH);
    const uint32_t unit = live ? static_cast<uint32_t>(e / CH) : 0u;
    const int tok = unit / G, gi = unit - tok * G;
    const int slot = a.slots[tok], pos = a.positions[tok];
    live = live && slot >= 0 && data_in_range(a.status, slot, a.num_slots, 701) &&
           data_in_range(a.status, pos, a.table_rows, 702);
    const int kind = gi < gq ? 0 : (gi < gq + gk ? 1 : 2);  // q, k, v
    const int h0 = (kind == 0 ? gi : (kind == 1 ? gi - gq : gi - gq - gk)) * HG, heads = kind == 0 ? a.H : a.Hkv;
    live = live && in_bounds(a.status, tok, a.T, 726) && in_bounds(a.status, h0, heads, 727);
    const size_t from = (static_cast<size_t>(tok) * heads + h0) * D + ch * 8;
    const size_t to = kind == 0 ? from : (static_cast<size_t>(live ? slot : 0) * heads + h0) * D + ch * 8;
    const __nv_bfloat16* src = (kind == 0 ? a.q : (kind == 1 ? a.k : a.v)) + from;
    __nv_bfloat16* dst = (kind == 0 ? a.q_out : (kind == 1 ? a.k_cache : a.v_cache)) + to;
    uint4 u1[HG], u2[HG];
#pragma unroll
    for (int k = 0; k < HG; ++k) {
      u1[k] = u2[k] = make_uint4(0, 0, 0, 0);
      if (live && h0 + k < heads) {
        u1[k] = *reinterpret_cast<const uint4*>(src + k * D);
        u2[k] = *reinterpret_cast<const uint4*>(src + k * D + D / 2);
      }
    }
    float c[8], s[8], w1[8], w2[8];
    load_turn(a.table, static_cast<size_t>(live ? pos : 0) * (D / 2) + ch * 8, c, s);
    if (NORM) {
      const W* w = static_cast<const W*>(kind == 0 ? a.wq : a.wk);
      load_w8(w, ch * 8, w1);
      load_w8(w, ch * 8 + D / 2, w2);
    }
#pragma unroll
    for (int k = 0; k < HG; ++k) {
      uint4 o1, o2;
      norm_rope_row<D, NORM>(u1[k], u2[k], w1, w2, c, s, a.eps, o1, o2);
      if (live && h0 + k < heads) {
        *reinterpret_cast<uint4*>(dst + k * D) = kind == 2 ? u1[k] : o1;
        *reinterpret_cast<uint4*>(dst + k * D + D / 2) = kind == 2 ? u2[k] : o2;
      }
    }
  }
}

// Blocks for n threads of work, at most `per_sm` an SM.
int blocks_for(long long n, int num_sms, int per_sm) {
  const long long b = (n + 255) / 256;
  const long long cap = static_cast<long long>(num_sms) * per_sm;
  return static_cast<int>(b < cap ? b : cap);
}

template <int D, typename W>
void fwd_launch(const QkNormArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int HG = 4;
  const long long n = static_cast<long long>(a.tokens) * ((a.H + HG - 1) / HG + (a.Hkv + HG - 1) / HG) * (D / 16);
  s2_qknorm_fwd_kernel<D, W, HG><<<blocks_for(n, num_sms, 16), 256, 0, stream>>>(a);
}

template <int D, typename W>
cudaError_t bwd_launch(QkNormArgs a, int num_sms, cudaStream_t stream) {
  constexpr int HG = 2;
  // blocks in proportion to the rows of either kind, at most 4 an SM in all (two
  // run at a time) and no more than the workspace holds
  const long long nq = static_cast<long long>(a.tokens) * ((a.H + HG - 1) / HG) * (D / 16);
  const long long nk = static_cast<long long>(a.tokens) * ((a.Hkv + HG - 1) / HG) * (D / 16);
  const long long bq = (nq + 255) / 256, bk = (nk + 255) / 256;
  const long long most = num_sms * 4 < kQkNormMaxBlocks ? num_sms * 4 : kQkNormMaxBlocks;
  if (bq + bk <= most) {
    a.blocks_q = static_cast<int>(bq);
    a.blocks = static_cast<int>(bq + bk);
  } else {
    const double part = static_cast<double>(nq) / static_cast<double>(nq + nk);
    const int share = static_cast<int>(part * static_cast<double>(most) + 0.5);
    a.blocks = static_cast<int>(most);
    a.blocks_q = share < 1 ? 1 : (share > a.blocks - 1 ? a.blocks - 1 : share);
  }
  prof_before(stream, kKernelQkNormBwd);
  s2_qknorm_bwd_kernel<D, W, HG><<<a.blocks, 256, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  prof_after(stream);
  if (e != cudaSuccess) return e;
  prof_before(stream, kKernelQkNormDw);
  e = launch_dependent(s2_qknorm_dw_kernel<D, W>, dim3(2 * D / 32), 1024, stream, a);
  prof_after(stream);
  return e;
}

template <int D, typename W>
void append_launch(const CacheAppendArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int HG = 4;
  const long long n = static_cast<long long>(a.T) * ((a.H + HG - 1) / HG + 2 * ((a.Hkv + HG - 1) / HG)) * (D / 16);
  const int grid = blocks_for(n, num_sms, 16);
  if (a.wq != nullptr)
    s2_cache_append_kernel<D, W, true, HG><<<grid, 256, 0, stream>>>(a);
  else
    s2_cache_append_kernel<D, W, false, HG><<<grid, 256, 0, stream>>>(a);
}

}  // namespace

cudaError_t launch_qknorm_fwd(const QkNormArgs& a, int D, int w_fp32, int num_sms, cudaStream_t stream) {
  prof_before(stream, kKernelQkNorm);
  if (D == 64)
    w_fp32 ? fwd_launch<64, float>(a, num_sms, stream) : fwd_launch<64, __nv_bfloat16>(a, num_sms, stream);
  else
    w_fp32 ? fwd_launch<128, float>(a, num_sms, stream) : fwd_launch<128, __nv_bfloat16>(a, num_sms, stream);
  const cudaError_t e = cudaGetLastError();
  prof_after(stream);
  return e;
}

cudaError_t launch_qknorm_bwd(const QkNormArgs& a, int D, int w_fp32, int num_sms, cudaStream_t stream) {
  if (D == 64)
    return w_fp32 ? bwd_launch<64, float>(a, num_sms, stream) : bwd_launch<64, __nv_bfloat16>(a, num_sms, stream);
  return w_fp32 ? bwd_launch<128, float>(a, num_sms, stream) : bwd_launch<128, __nv_bfloat16>(a, num_sms, stream);
}

cudaError_t launch_cache_append(const CacheAppendArgs& a, int D, int w_fp32, int num_sms, cudaStream_t stream) {
  prof_before(stream, kKernelCacheAppend);
  if (D == 64)
    w_fp32 ? append_launch<64, float>(a, num_sms, stream) : append_launch<64, __nv_bfloat16>(a, num_sms, stream);
  else
    w_fp32 ? append_launch<128, float>(a, num_sms, stream) : append_launch<128, __nv_bfloat16>(a, num_sms, stream);
  const cudaError_t e = cudaGetLastError();
  prof_after(stream);
  return e;
}

}  // namespace s2
