// Attention of new tokens over a paged cache on the tensor cores (tcgen05,
// TMEM accumulators, TMA-fed rings): one token, a chain or a tree of drafts for
// each request of a ragged batch.
//
//   o = softmax(q K^T / sqrt(D), masked) V,  lse = log sum exp (natural log)
//
// Token j of request i (rows cu[i] .. cu[i+1]) sees every key before ctx_i and,
// of the request's own new keys, those its mask names (bit j' = draft j'), or
// without masks the drafts up to itself.  Key p of request i is row p % bs of
// cache block block_table[i][p / bs].
//
// Rows.  The rep = H/Hkv query heads that share a kv head form one 128-row tile
// with floor(128 / rep) tokens: row = token * rep + head in group, which is the
// order a {64 columns, rep heads, tokens} TMA box lands in shared memory.  An
// item is two adjacent tiles (A, B) of one (request, kv head).
//
// Split.  One CTA per SM walks an equal run of units of 128 keys (s2_cache.cuh).
//
// Two ways through a segment keep both softmax warpgroups and the tensor core
// busy.  Paired (the item has tile B): every key tile feeds both query tiles,
// one load for 256 rows.  Alternating (few rows, tile A alone): warpgroup A
// takes the even and warpgroup B the odd key tiles of the same query tile, and
// A joins the two accumulators from TMEM at the end.  With few rows the kernel
// is bound by reading the cache; the padding of the 128-row tile is free there
// (1024 tensor cycles a 64 KB tile against some 2800 of HBM time).
//
// Warp roles (320 threads): warp 0 TMA producer (segments, Q ring, K/V ring, the
// pages of a tile loaded by one lane each), warp 1 UMMA issuer, warps 2-5 softmax A,
// warps 6-9 softmax B, one thread per query row.  P is rounded to bf16 for the
// product with V; its row sums, the maxima and O stay fp32.  Rows of V behind
// the last key may hold anything (stale cache rows): the product stops at the
// 16-key step that holds the last key, and the rows of that step behind it are
// zeroed in shared memory first, as are infinite and NaN values of drafts,
// which only the rows that see them may get.
//
// TMEM (512 columns): S_A [0,128), S_B [128,256) (P over their first 64
// columns), O_A [256, 256+D), O_B [384, 384+D).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "s2_cache.cuh"

namespace s2 {

namespace {

using namespace cache;

constexpr int kThreads = 320;
constexpr int kPair = 2 * kTile;  // rows of an item

template <int D>
struct TcCfg {
  static constexpr int NQ = D == 128 ? 2 : 4;       // Q ring
  static constexpr int NS = D == 128 ? 5 : 10;      // K/V ring
  static constexpr int NG = 4;                      // segment descriptions
  static constexpr int ATOM = kTile * 128;          // one 64-column slab of a 128-row tile
  static constexpr int TILE = kTile * D * 2;
  static constexpr int OFF_KV = NQ * TILE;
  static constexpr int SMEM = OFF_KV + NS * TILE + 1024;
  static constexpr uint32_t TM_O = 256, TM_OB = 384;
  static_assert(SMEM <= 232448 - 2048, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    s2_cache_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CacheAttnArgs a) {
  using C = TcCfg<D>;
  constexpr int NQ = C::NQ, NS = C::NS;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t bar_qfull[NQ], bar_qempty[NQ], bar_full[NS], bar_empty[NS], bar_s[2], bar_plo[2],
      bar_p[2], bar_o[2], bar_ofree[2], bar_mb, bar_drain, bar_gfull[C::NG], bar_gempty[C::NG];
  __shared__ Seg segs[C::NG];
  __shared__ uint32_t odd[C::NG];  // the segment's drafts hold infinite or NaN values
  __shared__ uint32_t tmem_slot, abort_flag;
  __shared__ long long sums[kThreads / 32];
  __shared__ Found found;
  __shared__ float b_m[kTile], b_l[kTile];  // alternating: warpgroup B's row maxima and sums

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  launch_dependents();
  if (tid < 3) tma_prefetch_desc(tid == 0 ? &tmQ : tid == 1 ? &tmK : &tmV);
  if (tid == 0) a.desc[blockIdx.x] = make_int4(0, -1, 0, 0);
  Run run;
  if (!locate<kThreads, kTile>(a, 2 * a.tpt, 1, sums, &found, run)) return;
  WaitCtx wc{&abort_flag, a.status, a.wait_limit_ns};
  const uint32_t sQ = smem_u32(smem);
  auto q_addr = [&](int s) { return sQ + s * C::TILE; };
  auto kv_addr = [&](int s) { return sQ + C::OFF_KV + s * C::TILE; };
  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < NQ; ++s) {
      mbar_init(smem_u32(&bar_qfull[s]), 1);
      mbar_init(smem_u32(&bar_qempty[s]), 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);
      mbar_init(smem_u32(&bar_empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar_s[i]), 1);
      mbar_init(smem_u32(&bar_plo[i]), 4);
      mbar_init(smem_u32(&bar_p[i]), 4);
      mbar_init(smem_u32(&bar_o[i]), 1);
      mbar_init(smem_u32(&bar_ofree[i]), 4);
    }
    for (int s = 0; s < C::NG; ++s) {
      mbar_init(smem_u32(&bar_gfull[s]), 1);
      mbar_init(smem_u32(&bar_gempty[s]), 9);  // the issuer and the softmax warps
    }
    mbar_init(smem_u32(&bar_mb), 4);
    mbar_init(smem_u32(&bar_drain), 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // The producer walks the segments and hands their descriptions over in a
  // ring; the other warps keep one until they are done with it (ng: how many
  // they have had).
  auto get_seg = [&](int ng, int where) {
    return warp_wait(smem_u32(&bar_gfull[ng % C::NG]), (ng / C::NG) & 1, wc, where);
  };
  auto put_seg = [&](int ng) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bar_gempty[ng % C::NG]));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    Seg sg;
    int qu = 0, L = 0;  // ring uses so far
    bool ok = true;
    const int page_rows = min(1 << a.bs_log2, kTile), page_log2 = min(a.bs_log2, 7);
    auto load_q = [&](int token) -> bool {
      const int s = qu % NQ, r = qu / NQ;
      if (r > 0 && !warp_wait(smem_u32(&bar_qempty[s]), (r - 1) & 1, wc, 110)) return false;
      if (elect_one()) {
        mbar_arrive_expect_tx(smem_u32(&bar_qfull[s]), a.tpt * a.rep * 128 * (D / 64));
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(q_addr(s) + c * C::ATOM, &tmQ, smem_u32(&bar_qfull[s]), c * 64, sg.kvh * a.rep,
                      in_bounds(a.status, token, a.T, 748) ? token : 0, 0);
      }
      __syncwarp();
      ++qu;
      return true;
    };
    // one lane per page; a block outside the cache reads as zeros (its row lies behind the tensor)
    auto load_kv = [&](const CUtensorMap* map, bool mine, int row) -> bool {
      const int s = L % NS, r = L / NS;
      if (r > 0 && !warp_wait(smem_u32(&bar_empty[s]), (r - 1) & 1, wc, 111)) return false;
      const int pages = __popc(__ballot_sync(0xffffffffu, mine));
      if (lane == 0) mbar_arrive_expect_tx(smem_u32(&bar_full[s]), pages * page_rows * 128 * (D / 64));
      __syncwarp();
      if (mine)
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(kv_addr(s) + c * C::ATOM + (lane << page_log2) * 128, map, smem_u32(&bar_full[s]), c * 64, sg.kvh,
                      row, 0);
      __syncwarp();
      ++L;
      return true;
    };
    for (int ng = 0; ok; ++ng) {
      const bool more = next_segment<kTile>(a, 2 * a.tpt, run, sg);
      if (!more) sg.tiles = -1;
      const int gs = ng % C::NG;
      if (ng >= C::NG && !(ok = warp_wait(smem_u32(&bar_gempty[gs]), (ng / C::NG - 1) & 1, wc, 112))) break;
      if (lane == 0) {
        segs[gs] = sg;
        odd[gs] = 0;
        mbar_arrive(smem_u32(&bar_gfull[gs]));
      }
      __syncwarp();
      if (!more) break;
      if (sg.tiles == 0) continue;
      ok = load_q(sg.row0 + sg.tok) && (sg.ntok <= a.tpt || load_q(sg.row0 + sg.tok + a.tpt));
      for (int i = 0; ok && i < sg.tiles; ++i) {
        const int key = (sg.kt0 + i) * kTile + (lane << page_log2);
        const bool mine = lane < (kTile >> page_log2) && key < sg.keys;
        int row = 0;
        if (mine) {
          const int blk = block_of(a, sg.ri, key);
          row = data_in_range(a.status, blk, a.num_blocks, 711) ? (blk << a.bs_log2) + (key & ((1 << a.bs_log2) - 1))
                                                                : a.num_blocks << a.bs_log2;
        }
        ok = load_kv(&tmK, mine, row) && load_kv(&tmV, mine, row);
      }
    }
    if (lane == 0) {
      // never leave copies in flight into shared memory: wait (bounded) for
      // the last fill of every slot -- always, since a consumer can give up
      // after this warp has issued its last copy
      for (int s = 0; s < NQ && s < qu; ++s) drain_wait(smem_u32(&bar_qfull[s]), ((qu - 1 - s) / NQ) & 1);
      for (int s = 0; s < NS && s < L; ++s) drain_wait(smem_u32(&bar_full[s]), ((L - 1 - s) / NS) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ UMMA issuer
    const uint32_t idS = make_idesc_bf16(128, kTile, 0, 0);  // Q K-major, K K-major
    const uint32_t idO = make_idesc_bf16(128, D, 0, 1);      // P from TMEM, V MN-major
    const uint64_t dQ0 = make_sdesc_sw128(q_addr(0), 16, 1024);
    const uint64_t dK0 = make_sdesc_sw128(kv_addr(0), 16, 1024);
    const uint64_t dV0 = make_sdesc_sw128(kv_addr(0), C::ATOM, 1024);
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) umma_commit(smem_u32(bar));
      __syncwarp();
    };
    auto wait_full = [&](int Lx) { return warp_wait(smem_u32(&bar_full[Lx % NS]), (Lx / NS) & 1, wc, 120); };
    auto issue_s = [&](int wg, int qs, int Lk) {
      tc_fence_after();
      const uint64_t dq = sdesc_advance(dQ0, qs * C::TILE);
      const uint64_t dk = sdesc_advance(dK0, (Lk % NS) * C::TILE);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::ATOM + (kk & 3) * 32;
          umma_ss(tmem + wg * 128, sdesc_advance(dq, off), sdesc_advance(dk, off), idS, kk > 0);
        }
        umma_commit(smem_u32(&bar_s[wg]));
      }
      __syncwarp();
    };
    int L = 0, qu = 0, np[2] = {0, 0}, nseg[2] = {0, 0};
    // O_wg (+)= P_wg V(load Lv), half h of the tile's keys, as far as there are
    // nk 16-key steps with a key; the second half completes the product (bar_o)
    auto issue_pv = [&](int wg, int Lv, int h, int nk, bool acc) {
      tc_fence_after();
      const uint64_t dv = sdesc_advance(dV0, (Lv % NS) * C::TILE);
      if (elect_one()) {
#pragma unroll
        for (int kq = 0; kq < kTile / 32; ++kq) {
          const int kk = h * (kTile / 32) + kq;
          if (kk < nk)
            umma_ts(tmem + (wg ? C::TM_OB : C::TM_O), tmem + wg * 128 + kk * 8, sdesc_advance(dv, kk * 2048), idO,
                    acc || kk > 0);
        }
        if (h == 1) umma_commit(smem_u32(&bar_o[wg]));
      }
      __syncwarp();
    };
    // step j of warpgroup wg: P V, keys 0..63 as soon as they are there
    auto pv = [&](int wg, int Lv, int j, int nk) -> bool {
      if (!warp_wait(smem_u32(&bar_plo[wg]), np[wg] & 1, wc, 122 + wg)) return false;
      if (j == 0 && nseg[wg] > 0 && !warp_wait(smem_u32(&bar_ofree[wg]), (nseg[wg] - 1) & 1, wc, 124 + wg)) return false;
      if (!wait_full(Lv)) return false;
      issue_pv(wg, Lv, 0, nk, j > 0);
      if (!warp_wait(smem_u32(&bar_p[wg]), np[wg] & 1, wc, 126 + wg)) return false;
      issue_pv(wg, Lv, 1, nk, true);
      ++np[wg];
      return true;
    };
    bool ok = true;
    for (int ng = 0; ok; ++ng) {
      if (!(ok = get_seg(ng, 128))) break;
      const Seg& sg = segs[ng % C::NG];
      const int n = sg.tiles, kt0 = sg.kt0, keys = sg.keys;
      const bool alt = sg.ntok <= a.tpt;
      put_seg(ng);
      if (n < 0) break;
      if (n == 0) continue;
      const int nA = alt ? (n + 1) / 2 : n, nB = alt ? n / 2 : n;
      const int qa = qu % NQ, qb = alt ? qa : (qu + 1) % NQ, L0 = L;
      // load of the K tile of step j (its V tile is the next load), and the
      // 16-key steps of its key tile that hold a key
      auto lk = [&](int wg, int j) { return L0 + (alt ? 4 * j + 2 * wg : 2 * j); };
      auto steps16 = [&](int wg, int j) {
        return (min(keys - (kt0 + (alt ? 2 * j + wg : j)) * kTile, kTile) + 15) >> 4;
      };
      ok = warp_wait(smem_u32(&bar_qfull[qa]), (qu / NQ) & 1, wc, 121) &&
           (alt || warp_wait(smem_u32(&bar_qfull[qb]), ((qu + 1) / NQ) & 1, wc, 121)) && wait_full(lk(0, 0));
      if (!ok) break;
      issue_s(0, qa, lk(0, 0));
      if (alt) commit(&bar_empty[lk(0, 0) % NS]);
      if (nB > 0) {
        if (alt && !(ok = wait_full(lk(1, 0)))) break;
        issue_s(1, qb, lk(1, 0));
        commit(&bar_empty[lk(1, 0) % NS]);
      }
      for (int j = 0; ok && j < nA; ++j) {
        if (!(ok = pv(0, lk(0, j) + 1, j, steps16(0, j)))) break;
        if (alt) commit(&bar_empty[(lk(0, j) + 1) % NS]);
        if (j + 1 < nA) {
          if (!(ok = wait_full(lk(0, j + 1)))) break;
          issue_s(0, qa, lk(0, j + 1));
          if (alt) commit(&bar_empty[lk(0, j + 1) % NS]);
        }
        if (j < nB) {
          if (!(ok = pv(1, lk(1, j) + 1, j, steps16(1, j)))) break;
          commit(&bar_empty[(lk(1, j) + 1) % NS]);
          if (j + 1 < nB) {
            if (alt && !(ok = wait_full(lk(1, j + 1)))) break;
            issue_s(1, qb, lk(1, j + 1));
            commit(&bar_empty[lk(1, j + 1) % NS]);
          }
        }
      }
      if (!ok) break;
      commit(&bar_qempty[qa]);
      if (!alt) commit(&bar_qempty[qb]);
      qu += alt ? 1 : 2;
      L = L0 + 2 * n;
      ++nseg[0];
      nseg[1] += nB > 0;
    }
    // every issued UMMA completes before TMEM is released
    if (elect_one()) {
      umma_commit(smem_u32(&bar_drain));
      drain_wait(smem_u32(&bar_drain), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int wg = (warp - 2) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + wg * 128;
    const uint32_t tO = tS + C::TM_O;  // O_B lies 128 columns behind O_A, as S_B behind S_A
    const float sl2 = a.scale_log2;
    int ns = 0, nsb = 0, nmb = 0, L = 0;  // phases so far (S and P V go together; A counts B's); K/V ring loads consumed
    bool ok = true;
    for (int ng = 0; ok; ++ng) {
      if (!(ok = get_seg(ng, 129))) break;
      const Seg& sg = segs[ng % C::NG];  // read where it is needed: registers are short
      const int n = sg.tiles;
      if (n < 0) break;
      const bool alt = sg.ntok <= a.tpt;
      const int steps = alt ? (n + 1 - wg) / 2 : n, ctx = sg.ctx;
      L += 2 * n;
      // the warp has a live row
      const bool busy = quarter * 32 < (alt || wg == 0 ? min(sg.ntok, a.tpt) : sg.ntok - a.tpt) * a.rep;
      float m_run = kFloor, l_run = 0.f;
      int key0 = (sg.kt0 + (alt ? wg : 0)) * kTile;
      for (int j = 0; j < steps; ++j, key0 += alt ? 2 * kTile : kTile) {
        ok = warp_wait(smem_u32(&bar_s[wg]), ns & 1, wc, 130);
        if (!ok) break;
        ++ns;
        const bool edge = key0 + kTile > ctx;  // drafts, or keys behind the last, in this tile
        if (edge && (alt || wg == 0)) {
          const bool hides = a.mask != nullptr || sg.keys - ctx > 1;  // some row may not see some draft
          const int valid = min(sg.keys - key0, kTile), drafts = hides ? valid - max(ctx - key0, 0) : 0;
          if ((valid & 15) != 0 || drafts > 0) {
            // (After the wait for S: the slot's earlier tile has been used by
            // then, so this wait cannot mistake its phase.)
            const int Lv = L - 2 * n + (alt ? 4 * j + 2 * wg : 2 * j) + 1;
            ok = warp_wait(smem_u32(&bar_full[Lv % NS]), (Lv / NS) & 1, wc, 133);
            if (!ok) break;
            clean_v<D>(kv_addr(Lv % NS), valid, drafts, row, odd[ng % C::NG]);
          }
        }
        if (!busy) {  // no live row: only the protocol
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bar_plo[wg]));
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bar_p[wg]));
          continue;
        }
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, sr[c]);
        tmem_wait_ld();
        if (edge) {
          // (the row's token is worked out here, for the one or two such tiles of a segment)
          mask_row128(a, sg, key0, sg.tok + (alt || wg == 0 ? 0 : a.tpt) + row / a.rep, sr);
        }
        float m4[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            m4[u] = fmax3(m4[u], __uint_as_float(sr[c >> 5][(c & 31) + 2 * u]),
                          __uint_as_float(sr[c >> 5][(c & 31) + 2 * u + 1]));
        }
        const float mx = fmax3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * sl2;
        float alpha = 1.f;
        bool resc = false;
        if (j == 0) {
          m_run = fmaxf(mx, kFloor);
        } else if (mx > m_run + 8.f) {  // P stays below 2^8: O is rescaled rarely
          alpha = ex2_approx(m_run - mx);
          m_run = mx;
          resc = true;
        }
        uint32_t pk[16];
        float rs = softmax_row32(sr[0], sl2, m_run, pk);
        tmem_st16(tS, pk);
        rs += softmax_row32(sr[1], sl2, m_run, pk);
        tmem_st16(tS + 16, pk);
        if (__any_sync(0xffffffffu, resc)) {
          // O holds P V up to the previous step once that UMMA has completed
          ok = warp_wait(smem_u32(&bar_o[wg]), ns & 1, wc, 131);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(tO + c * 16, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16(tO + c * 16, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_plo[wg]));
        rs += softmax_row32(sr[2], sl2, m_run, pk);
        tmem_st16(tS + 32, pk);
        rs += softmax_row32(sr[3], sl2, m_run, pk);
        tmem_st16(tS + 48, pk);
        l_run = l_run * alpha + rs;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_p[wg]));
      }
      if (!ok) break;
      const int nB = alt ? n / 2 : n;
      nsb += nB;  // warpgroup B's products, which A waits for when it joins them
      // ---------------------------------------------------------- epilogue
      int erow = row;
      asm volatile("" : "+r"(erow));  // (computed here again rather than held through the loop)
      const bool second = wg == 1 && !alt;  // this warpgroup worked on tile B
      const int jt = erow / a.rep, gtok = sg.row0 + sg.tok + (second ? a.tpt : 0) + jt;
      const int head = sg.kvh * a.rep + erow - jt * a.rep;
      const bool live = jt < (second ? sg.ntok - a.tpt : min(sg.ntok, a.tpt)) && row_in(a, gtok, head, 749);
      // where the row goes: o and lse, or this CTA's part (0: the item began before, 1: it begins here)
      float* part = Part<kPair, D>::at(a, blockIdx.x, sg.first);
      const int prow = (second ? kTile : 0) + row;
      __nv_bfloat16* orow = a.o + (static_cast<size_t>(gtok) * a.H + head) * D;
      auto finish = [&](float m, float l) {
        if (!live) return;
        if (sg.whole) {
          a.lse[static_cast<size_t>(head) * a.T + gtok] = lse_of(m, l);
        } else {
          part[kPair * D + prow] = m;
          part[kPair * (D + 1) + prow] = l;
        }
        if (odd[ng % C::NG]) add_odd<D>(a, sg, gtok, orow, part + prow * D);
      };
      if (steps > 0) {
        ok = warp_wait(smem_u32(&bar_o[wg]), (ns - 1) & 1, wc, 132);
        if (!ok) break;
        tc_fence_after();
      }
      if (alt && wg == 1) {
        if (steps > 0) {  // hand the row's statistics to warpgroup A, which reads O_B out of TMEM
          b_m[row] = m_run;
          b_l[row] = l_run;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bar_mb));
        }
      } else if (alt && nB > 0) {
        ok = warp_wait(smem_u32(&bar_mb), nmb & 1, wc, 134) &&
             warp_wait(smem_u32(&bar_o[1]), (nsb - 1) & 1, wc, 135);
        if (!ok) break;
        ++nmb;
        tc_fence_after();
        const float mb = b_m[row], lb = b_l[row], m = fmaxf(m_run, mb);
        const float fa = ex2_approx(m_run - m), fb = ex2_approx(mb - m), l = fa * l_run + fb * lb;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (busy) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t va[32], vb[32];
            tmem_ld32(tO + c * 32, va);
            tmem_ld32(tO + 128 + c * 32, vb);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              va[i] = __float_as_uint(fmaf(fa, __uint_as_float(va[i]), fb * __uint_as_float(vb[i])));
            if (live) store_o32(orow + c * 32, part + prow * D + c * 32, sg.whole, va, inv);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bar_ofree[0]));
          mbar_arrive(smem_u32(&bar_ofree[1]));
        }
        finish(m, l);
      } else {
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
        if (steps > 0) {
          if (busy) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(tO + c * 32, v);
              tmem_wait_ld();
              if (live) store_o32(orow + c * 32, part + prow * D + c * 32, sg.whole, v, inv);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bar_ofree[wg]));
        }
        finish(m_run, l_run);
      }
      if (sg.first && !sg.whole && wg == 0 && row == 0 && in_bounds(a.status, sg.last_cta, gridDim.x, 750))
        // join work: the parts lie in CTAs blockIdx.x .. last_cta
        a.desc[blockIdx.x] = join_work(sg);
      put_seg(ng);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t tc_launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CacheAttnArgs& a,
                      int grid, cudaStream_t stream) {
  const cudaError_t ea =
      cudaFuncSetAttribute(s2_cache_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcCfg<D>::SMEM);
  if (ea != cudaSuccess) return ea;
  prof_before(stream, kKernelCacheAttn);
  s2_cache_tc_kernel<D><<<grid, kThreads, TcCfg<D>::SMEM, stream>>>(tq, tk, tv, a);
  cudaError_t e = cudaGetLastError();
  prof_after(stream);
  if (e != cudaSuccess) return e;
  return launch_join<kPair, kTile, D, 1, 2>(a, grid, stream);
}

}  // namespace

cudaError_t launch_cache_tc(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CacheAttnArgs& a,
                            int D, int grid, cudaStream_t stream) {
  return D == 64 ? tc_launch<64>(tq, tk, tv, a, grid, stream) : tc_launch<128>(tq, tk, tv, a, grid, stream);
}

}  // namespace s2
