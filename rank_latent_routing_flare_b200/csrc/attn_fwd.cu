// Exact softmax attention, forward, on tcgen05: per query row i
//
//   x_ij = score of <q_i, k_j> (scaled, capped, biased), in log2 units
//   Y_i = sum_j 2^(x_ij - m_i) v_j / l_i,  l_i = sum_j 2^(x_ij - m_i)
//
// over the interval [lo_i, hi_i) of keys that the masks leave the row, with
// the running reference m_i and sum l_i of an online softmax.
//
// A CTA owns two tiles of 128 query rows of one head and one range of key
// tiles of KT keys; each query tile belongs to one warpgroup (thread <-> TMEM
// lane <-> row).  Per key tile and query tile w:
//   S_w = Q_w K^T        UMMA 128 x KT, fp32 in TMEM
//   P_w = 2^(x - m)      softmax threads, bf16 over the columns of S_w
//   O_w += P_w V         UMMA, P_w read from TMEM
// One thread issues the MMAs in the order P_0 V, S_0 (next tile), P_1 V, S_1
// (next tile): the tensor pipe runs them in order, so S_w may overwrite P_w
// right behind the product that reads it, and one warpgroup's exponentials
// run under the other's products.  Both query tiles read each K and V tile
// from shared memory once.  O_w is rescaled only when a row's maximum has
// grown by more than 2^8 over its reference (weights then reach 2^8, which
// bf16 and the fp32 sums hold as well as 1): S_w complete implies the
// products before it are, so the softmax threads rescale TMEM themselves.
//
// Tiles outside [lo of the first row, hi of the last) are not visited; the
// interval is tested per element only in tiles that some row of the warp does
// not see whole.  A weight of 0 does not erase a NaN in V, so rows of V that
// no row of the CTA sees (padding, other documents, slots of a cache behind
// the newest token) are zeroed in shared memory by the softmax threads before
// the product.
//
// D = 128, and capped or biased scores: KT = 128, 512 TMEM columns, one CTA per
// SM whose softmax threads take over most of its registers.  Plain scores of D
// <= 64: KT = 64 and 256 columns let two CTAs share an SM.  Measured on 2 x 16
// heads x 4096^2, D = 64: plain 228 us (one CTA: 254), capped 300 (two CTAs,
// which spill: 364), biased 286 (337); D = 128: plain 289, capped 332.
#include <utility>

#include "attn_common.cuh"
#include "ops_internal.h"

namespace flare {
namespace {

// MOD: 0 plain scores, 1 capped, 2 with a distance bias (and capped if p.cap > 0).
template <int D, int MOD>
struct FwdCfg {
  using Tile = RowTile<D>;
  static constexpr bool WIDE = D == 128 || MOD != 0;
  static constexpr int NQ = 2;                            // query tiles, and softmax warpgroups, of a CTA
  static constexpr int KT = WIDE ? 128 : 64;
  static constexpr int QT = kAttnQTile;
  static constexpr int CTAS = WIDE ? 1 : 2;
  static constexpr int NST = D == 128 ? 2 : D == 64 ? 4 : 6;
  static constexpr int Q_B = Tile::bytes(QT), KV_B = Tile::bytes(KT);
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + NQ * Q_B;
  static constexpr int OFF_V = OFF_K + NST * KV_B;
  static constexpr int OFF_BAR = OFF_V + NST * KV_B;
  static constexpr int N_BAR = 2 + 2 * NST + 2 + 2 + 2 + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * N_BAR;
  static constexpr int BYTES = OFF_MISC + 32 + 4 * NST;
  // a cluster's partial outputs, over the operands, and their log2 sums
  static constexpr int PART = D + 4, OFF_LSE = NQ * QT * PART * 4;
  static_assert(OFF_LSE + NQ * QT * 4 <= OFF_BAR, "partial results fit over the operands");
  static constexpr uint32_t COL_S = 0, COL_O = NQ * KT;
  static constexpr uint32_t TMEM_COLS = COL_O + NQ * D <= 256 ? 256 : 512;
  // Warps: softmax (four per query tile), loads, MMAs.  One CTA an SM:
  // two more fill a third warpgroup, which gives the softmax threads its
  // registers (168 a thread at launch).
  static constexpr int LOADS = 4 * NQ, MMAS = 4 * NQ + 1, THREADS = WIDE ? 384 : 32 * (4 * NQ + 2);
  static constexpr int LESS = 56, MORE = 224;
  static_assert(256 * MORE + 128 * LESS <= 384 * 168, "register split");
  static_assert(COL_O + NQ * D <= TMEM_COLS && TMEM_COLS * CTAS <= 512, "TMEM columns");
  static_assert(KV_B % 1024 == 0 && Q_B % 1024 == 0, "tiles hold whole swizzle atoms");
  static_assert(CTAS * (BYTES + 2048) <= 228 * 1024, "shared memory");
};

// Key tiles [a, b) that rows [r0, r0 + 128) see.
__device__ __forceinline__ int2 tile_range(const BatchMask& m, int r0, int KT) {
  const int r1 = min(r0 + kAttnQTile, m.qlen);
  if (r0 >= r1) return make_int2(0, 0);
  const int lo = row_interval(m, r0).x, hi = row_interval(m, r1 - 1).y;
  return lo < hi ? make_int2(lo / KT, (hi + KT - 1) / KT) : make_int2(0, 0);
}

__device__ __forceinline__ void unpair(uint64_t v, uint32_t& a, uint32_t& b) {
  float x, y;
  f2_unpack(v, x, y);
  a = __float_as_uint(x);
  b = __float_as_uint(y);
}
// -inf outside columns [first, last).
template <int N>
__device__ __forceinline__ void hide(uint32_t (&s)[N], int first, int last) {
#pragma unroll
  for (int c = 0; c < N; c += 32) {
    const uint32_t bits = column_bits(first, last, c);
#pragma unroll
    for (int k = 0; k < 32; ++k) s[c + k] = bits & (1u << k) ? s[c + k] : 0xFF800000u;
  }
}
// Raw products to capped scores in log2 units, + c.
template <int N>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[N], const ScoreOps& ops, bool small, float c) {
  if (small) {
    const uint64_t c2 = f2_dup(c);
#pragma unroll
    for (int k = 0; k < N; k += 2) unpair(ops.poly(f2(s[k], s[k + 1]), c2), s[k], s[k + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = __float_as_uint(fmaf(ops.tanh_any(as_f(s[k])), ops.out, c));
  }
}
// s c2 minus slope2 |d - k| for column k.  Where every row of the warp stands
// behind (side 1) or before (-1) all keys of the tile the bias is linear in k:
// anchored every 16 columns and stepped in between, two columns an instruction.
template <int N>
__device__ __forceinline__ void bias_scores(uint32_t (&s)[N], float c2, float d, float slope2, int side) {
  const uint64_t c = f2_dup(c2);
  if (side != 0) {
    const float g = side > 0 ? -slope2 : slope2;
    const uint64_t step = f2_dup(-2.f * g);
#pragma unroll
    for (int k = 0; k < N; k += 16) {
      uint64_t b = f2_pack(g * (d - k), g * (d - (k + 1)));
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        unpair(f2_fma(f2(s[k + i], s[k + i + 1]), c, b), s[k + i], s[k + i + 1]);
        b = f2_add(b, step);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = __float_as_uint(fmaf(as_f(s[k]), c2, -slope2 * fabsf(d - k)));
  }
}
// Weights 2^(x - base) of a row's N columns, x = s c2 (RAW) or s, stored as
// bf16 pairs from TMEM column `col` on; returns their sum.
template <int N, bool RAW>
__device__ __forceinline__ float weights(const uint32_t (&s)[N], float c2, float base, uint32_t col) {
  const uint64_t c = f2_dup(c2), nb = f2_dup(-base);
  uint64_t sum0 = f2_dup(0.f), sum1 = sum0;
#pragma unroll
  for (int k = 0; k < N; k += 32) {
    uint32_t pk[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const uint64_t x = f2(s[k + 2 * q], s[k + 2 * q + 1]);
      float p0, p1;
      ex2_pair(RAW ? f2_fma(x, c, nb) : f2_add(x, nb), p0, p1);
      if (q & 1) sum1 = f2_add(sum1, f2_pack(p0, p1));
      else sum0 = f2_add(sum0, f2_pack(p0, p1));
      pk[q] = pack_bf16x2(p0, p1);
    }
    tmem_st16(col + k / 2, pk);
  }
  float a, b;
  f2_unpack(f2_add(sum0, sum1), a, b);
  return a + b;
}
// As weights<N, true>, with a bias linear in the column (see bias_scores).
template <int N>
__device__ __forceinline__ float biased_weights(const uint32_t (&s)[N], float c2, float base, float d, float slope2, int side,
                                                uint32_t col) {
  const uint64_t c = f2_dup(c2);
  const float g = side > 0 ? -slope2 : slope2;
  const uint64_t step = f2_dup(-2.f * g);
  uint64_t sum0 = f2_dup(0.f), sum1 = sum0;
#pragma unroll
  for (int k = 0; k < N; k += 32) {
    uint32_t pk[16];
    uint64_t b;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      if (q % 8 == 0) b = f2_pack(fmaf(g, d - (k + 2 * q), -base), fmaf(g, d - (k + 2 * q + 1), -base));
      float p0, p1;
      ex2_pair(f2_fma(f2(s[k + 2 * q], s[k + 2 * q + 1]), c, b), p0, p1);
      b = f2_add(b, step);
      if (q & 1) sum1 = f2_add(sum1, f2_pack(p0, p1));
      else sum0 = f2_add(sum0, f2_pack(p0, p1));
      pk[q] = pack_bf16x2(p0, p1);
    }
    tmem_st16(col + k / 2, pk);
  }
  float x, y;
  f2_unpack(f2_add(sum0, sum1), x, y);
  return x + y;
}
// As weights<N, true>, for capped scores of raw products: tanh and the shift
// by the base in one polynomial.  Needs small.  MASKED: 0 outside columns [first, last).
template <int N, bool MASKED>
__device__ __forceinline__ float capped_weights(const uint32_t (&s)[N], const ScoreOps& ops, float base, int first, int last,
                                                uint32_t col) {
  const uint64_t nb = f2_dup(-base);
  uint64_t sum0 = f2_dup(0.f), sum1 = sum0;
#pragma unroll
  for (int k = 0; k < N; k += 32) {
    uint32_t pk[16];
    const uint32_t bits = MASKED ? column_bits(first, last, k) : ~0u;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      float p0, p1;
      ex2_pair(ops.poly(f2(s[k + 2 * q], s[k + 2 * q + 1]), nb), p0, p1);
      if (MASKED) {
        p0 = bits & (1u << (2 * q)) ? p0 : 0.f;
        p1 = bits & (2u << (2 * q)) ? p1 : 0.f;
      }
      if (q & 1) sum1 = f2_add(sum1, f2_pack(p0, p1));
      else sum0 = f2_add(sum0, f2_pack(p0, p1));
      pk[q] = pack_bf16x2(p0, p1);
    }
    tmem_st16(col + k / 2, pk);
  }
  float a, b;
  f2_unpack(f2_add(sum0, sum1), a, b);
  return a + b;
}

template <int D, int MOD>
__global__ void __launch_bounds__(FwdCfg<D, MOD>::THREADS, FwdCfg<D, MOD>::CTAS)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const AttnParams p) {
  using Cfg = FwdCfg<D, MOD>;
  using Tile = RowTile<D>;
  constexpr int KT = Cfg::KT, QT = Cfg::QT, NST = Cfg::NST, NQ = Cfg::NQ;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = sm + Cfg::OFF_Q;
  uint8_t* sk = sm + Cfg::OFF_K;
  uint8_t* sv = sm + Cfg::OFF_V;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + Cfg::OFF_BAR);   // [2]
  uint64_t* kv_full = q_full + 2;                                     // [NST]
  uint64_t* kv_empty = kv_full + NST;                                 // [NST] products of the tile done
  uint64_t* s_full = kv_empty + NST;                                  // [2] scores of the next tile ready
  uint64_t* p_full = s_full + 2;                                      // [2] weights stored (one arrive per warp)
  uint64_t* o_full = p_full + 2;                                      // [2] last product done
  uint64_t* all_done = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Cfg::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(sm + Cfg::OFF_MISC + 4);
  volatile int* range = reinterpret_cast<volatile int*>(sm + Cfg::OFF_MISC + 8);       // [6]
  volatile int* last_load = reinterpret_cast<volatile int*>(sm + Cfg::OFF_MISC + 32);  // [NST]

  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int BH = p.B * p.Hq, n_qt = gridDim.x / BH;
  // the last query tiles see the most keys under a causal mask: first
  const int qt = n_qt - 1 - static_cast<int>(blockIdx.x) / BH, bh = static_cast<int>(blockIdx.x) % BH;
  const int b = bh / p.Hq, h = bh % p.Hq, hk = h / p.G;
  const int q0 = qt * NQ * QT, split = blockIdx.y;
  const BatchMask mask = batch_mask(p.mask, b);

  // The error word is clear before any wait can expire (seconds from now).
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 4) p.err[threadIdx.x] = 0u;
  if (threadIdx.x < NQ) {
    const int2 r = tile_range(mask, q0 + threadIdx.x * QT, KT);
    range[2 * threadIdx.x] = r.x;
    range[2 * threadIdx.x + 1] = r.y;
  }
  if (threadIdx.x == 32) {   // the keys from the first to the last that a row of the CTA sees
    const int r1 = min(q0 + NQ * QT, mask.qlen);
    range[4] = q0 < r1 ? row_interval(mask, q0).x : 0;
    range[5] = q0 < r1 ? row_interval(mask, r1 - 1).y : 0;
  }
  if (threadIdx.x == 64) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(o_full + i, 1);
    }
    for (int i = 0; i < NST; ++i) {
      mbar_init(kv_full + i, 1);
      mbar_init(kv_empty + i, 1);
      last_load[i] = -1;
    }
    mbar_init(all_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == Cfg::MMAS) {
    tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{p.err, abort_flag, p.timeout_ns};

  // this split's key tiles [jlo, jhi), taken in steps n = 0, 1, ...: from the
  // last one down under a distance bias, whose rows then meet their nearest
  // keys early and raise their reference no more (a causal mask puts those
  // last).  Each query tile takes part in steps [a, e).
  int a[2] = {range[0], range[2]}, e[2] = {range[1], range[3]};
  int jlo, jhi;
  {
    const bool live0 = a[0] < e[0], live1 = a[1] < e[1];
    jlo = live0 && live1 ? min(a[0], a[1]) : live0 ? a[0] : a[1];
    jhi = live0 && live1 ? max(e[0], e[1]) : live0 ? e[0] : e[1];
    const int per = (jhi - jlo + p.splits - 1) / p.splits;
    jlo = min(jhi, jlo + split * per);
    jhi = min(jhi, jlo + per);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int first = max(a[w], jlo), end = min(e[w], jhi);
      a[w] = MOD == 2 ? jhi - end : first - jlo;
      e[w] = MOD == 2 ? jhi - first : end - jlo;
      if (a[w] >= e[w]) a[w] = e[w] = 0;
    }
  }
  const int ntiles = jhi - jlo;
  auto key0 = [&](int n) { return (MOD == 2 ? jhi - 1 - n : jlo + n) * KT; };   // first key of step n

  if (warp >= Cfg::LOADS) {
    if constexpr (Cfg::WIDE) setmaxnreg_dec<Cfg::LESS>();
    if (warp == Cfg::LOADS) {
      // ------------------------------------------------------------ loads
      if (lane == 0 && ntiles > 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        for (int w = 0; w < NQ; ++w) {
          mbar_arrive_expect_tx(q_full + w, Cfg::Q_B);   // rows behind the tensor's last come as zeros
          Tile::load(sq + w * Cfg::Q_B, &tm_q, q_full + w, q0 + w * QT, h, b, QT);
        }
        for (int n = 0; n < ntiles; ++n) {
          const int st = n % NST;
          if (n >= NST && !mbar_wait(kv_empty + st, (n / NST - 1) & 1, wc)) break;
          mbar_arrive_expect_tx(kv_full + st, 2 * Cfg::KV_B);
          Tile::load(sk + st * Cfg::KV_B, &tm_k, kv_full + st, key0(n), hk, b, KT);
          Tile::load(sv + st * Cfg::KV_B, &tm_v, kv_full + st, key0(n), hk, b, KT);
          last_load[st] = n;
        }
      }
    } else if (warp == Cfg::MMAS) {
      // ------------------------------------------------------------ MMAs
      if (ntiles > 0) {   // the whole warp, converged
        const uint32_t idesc_s = idesc_bf16_f32(128, KT, false, false);
        const uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
        const uint64_t q_desc = Tile::desc_k(sq), k_desc = Tile::desc_k(sk), v_desc = Tile::desc_mn(sv, KT);
        // scores of tile n, once it has landed
        auto issue_s = [&](int w, int n) -> bool {
          const int st = n % NST;
          if (!mbar_wait_warp(kv_full + st, (n / NST) & 1, wc)) return false;
          tc_fence_after();
          const uint64_t qd = q_desc + static_cast<uint64_t>((w * Cfg::Q_B) >> 4);
          const uint64_t kd = k_desc + static_cast<uint64_t>((st * Cfg::KV_B) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_ss(tmem + Cfg::COL_S + w * KT, qd + Tile::kstep_k(kk, QT), kd + Tile::kstep_k(kk, KT), idesc_s,
                      kk > 0 ? 1u : 0u);
            umma_commit(s_full + w);
          }
          __syncwarp();
          return true;
        };
        bool ok = mbar_wait_warp(q_full, 0, wc) && mbar_wait_warp(q_full + 1, 0, wc);
        int used[2] = {0, 0};
#pragma unroll
        for (int w = 0; w < NQ; ++w)
          if (ok && a[w] < e[w] && a[w] == 0) ok = issue_s(w, 0);
        for (int n = 0; ok && n < ntiles; ++n) {
          const int st = n % NST;
#pragma unroll
          for (int w = 0; w < NQ; ++w) {
            if (ok && n >= a[w] && n < e[w]) {
              ok = mbar_wait_warp(p_full + w, used[w]++ & 1, wc);
              tc_fence_after();
              const uint64_t vd = v_desc + static_cast<uint64_t>((st * Cfg::KV_B) >> 4);
              if (ok && elect_one()) {
#pragma unroll
                for (int ks = 0; ks < KT / 16; ++ks)
                  umma_ts(tmem + Cfg::COL_O + w * D, tmem + Cfg::COL_S + w * KT + ks * 8, vd + ks * Tile::KSTEP_MN,
                          idesc_o, (n > a[w] || ks > 0) ? 1u : 0u);
                if (n + 1 == e[w]) umma_commit(o_full + w);
              }
              __syncwarp();
            }
            if (ok && n + 1 >= a[w] && n + 1 < e[w]) ok = issue_s(w, n + 1);
          }
          // a tile between the two ranges (documents can leave it out): its
          // copy lands before its stage is given back
          if (ok && (n < a[0] || n >= e[0]) && (n < a[1] || n >= e[1])) ok = mbar_wait_warp(kv_full + st, (n / NST) & 1, wc);
          if (elect_one()) umma_commit(kv_empty + st);
          __syncwarp();
        }
        if (elect_one()) umma_commit(all_done);   // every MMA issued above is done
        __syncwarp();
        mbar_wait_drain(all_done, 0, p.timeout_ns);
        __syncwarp();
      }
    }
  } else {
    if constexpr (Cfg::WIDE) setmaxnreg_inc<Cfg::MORE>();
    // ------------------------------------------------------------ softmax
    const int w = warp >> 2, wq = warp & 3;
    const int tid = threadIdx.x & 127;              // row of the tile; also the key whose V row it may zero
    const int row = q0 + w * QT + tid;
    const int2 iv = row < p.mask.Nq ? row_interval(mask, row) : make_int2(0, 0);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t col_s = lane_base + Cfg::COL_S + w * KT, col_o = lane_base + Cfg::COL_O + w * D;
    const ScoreOps ops(p.scale, p.cap, true);
    const bool capped = MOD == 1 || (MOD == 2 && p.cap > 0.f);
    const float slope2 = MOD == 2 ? p.slopes[h] * kLog2e : 0.f;
    const int pos = bias_position(mask, row, iv);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const int a_w = w ? a[1] : a[0], n_w = (w ? e[1] : e[0]) - a_w;
    const int seen0 = range[4], seen1 = range[5];
    for (int it = 0; it < n_w; ++it) {
      const int n = a_w + it, k0 = key0(n), st = n % NST;
      // the V row this thread answers for: a key that no row of the CTA sees
      bool dead = false;
      if (KT == 128 || tid < KT) {
        const int key = k0 + tid;
        dead = (key < seen0 || key >= seen1) && key < mask.nk;
        if (mask.doc && key < mask.nk) {
          const int2 d = mask.doc[key];
          dead |= d.x == d.y;
        }
      }
      if (!mbar_wait_warp(s_full + w, it & 1, wc)) { ok = false; break; }
      tc_fence_after();
      uint32_t s[KT];
      tmem_ld_cols<KT>(col_s, s);
      tmem_wait_ld();
      regs_loaded(s);
      const bool masked = !__all_sync(~0u, iv.x <= k0 && iv.y >= k0 + KT);   // some row does not see the whole tile
      const int first = iv.x - k0, last = iv.y - k0;
      // the row's maximum, in log2 units; scores that need more than a scale
      // and a shift replace the products here
      float mx;
      bool small = false;
      enum { kExact, kLinear, kNone } how = kExact;   // MOD 2: scores in place, bias to be added, weights all 0
      int linear_side = 0;
      if (MOD == 0) {
        if (masked) hide<KT>(s, first, last);
        mx = max_of(s) * ops.c2;
      } else if (MOD == 1) {
        // tanh grows with its argument: the maximum takes it once.  D <= 64:
        // hidden columns count too (under a cap of up to 55 they lie at most
        // 2^37 above 1, half the cap, and the row's own keys at least 2^-80, which
        // leaves weights of 2^-117 to fp32 and bf16) and get their zeros behind
        // the exponential: the same 12 documents in 8192 keys, a whole call, 205
        // -> 190 us.  A row's largest weight is then no exact 1 and is rounded to
        // bf16 like the others: relative error of Y 0.0018 -> 0.0021, of which
        // its own rounding is 0.0016.  At D = 128 the second body costs more than
        // it saves (prefixes 208 -> 215).
        mx = max_of(s);
        const bool poly = __all_sync(~0u, ops.small(fmaxf(mx, -min_of(s))));
        small = poly && (!masked || (D < 128 && ops.out <= 80.f));
        if (!small) {
          cap_scores<KT>(s, ops, poly, 0.f);
          if (masked) hide<KT>(s, first, last);
          mx = max_of(s);
        } else {
          mx = ops.capped(mx);
        }
      } else {
        if (capped) cap_scores<KT>(s, ops, __all_sync(~0u, ops.small(fmaxf(max_of(s), -min_of(s)))), 0.f);
        const int side = __all_sync(~0u, pos >= k0 + KT - 1) ? 1 : __all_sync(~0u, pos <= k0) ? -1 : 0;
        const float c = capped ? 1.f : ops.c2;
        // A tile that every row sees, all on one side: no score is above the
        // largest product with the smallest distance's bias (a negative
        // slope's largest).  The bound serves as the maximum where it is at
        // most 2^64 above it (`slack`); the row's sum is then at least
        // 2^-slack of the reference, and weights below 2^-64 of that change
        // no fp32 sum: a tile of such weights gets zeros (but a NaN is kept).
        if (side != 0 && !masked) {
          const int near = side > 0 ? pos - (k0 + KT - 1) : k0 - pos;
          mx = fmaf(max_of<KT, true>(s), c, -slope2 * static_cast<float>(slope2 >= 0.f ? near : near + KT - 1));
          const float slack = fabsf(slope2) * (KT - 1);
          const bool steep = slack > 64.f;                    // references of this row are maxima
          how = it > 0 && __all_sync(~0u, mx < m - (steep ? 64.f : 64.f + slack)) ? kNone : steep ? kExact : kLinear;
        }
        if (how == kExact) {
          bias_scores<KT>(s, c, static_cast<float>(pos - k0), slope2, side);
          if (masked) hide<KT>(s, first, last);
          mx = max_of(s);
        }
        linear_side = side;
      }
      if (MOD == 2 && how == kNone) {
        // the reference stays
      } else if (it == 0) {
        m = mx;
      } else if (__any_sync(~0u, mx > m + 8.f)) {
        const float m_new = fmaxf(m, mx);
        const float fac = m == -INFINITY ? 0.f : ex2_mufu(m - m_new);
        m = m_new;
        l *= fac;
#pragma unroll
        for (int k = 0; k < D; k += 16) {
          uint32_t o[16];
          tmem_ld16(col_o + k, o);
          tmem_wait_ld();
          regs_loaded(o);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(as_f(o[i]) * fac);
          tmem_st16(col_o + k, o);
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      float sum = 0.f;
      if (MOD == 2 && how == kNone) {
        uint32_t none[16] = {};
#pragma unroll
        for (int k = 0; k < KT; k += 32) tmem_st16(col_s + k / 2, none);
      } else if (MOD == 2 && how == kLinear) {
        sum = biased_weights<KT>(s, capped ? 1.f : ops.c2, base, static_cast<float>(pos - k0), slope2, linear_side, col_s);
      } else if (MOD == 1 && small) {
        if (D < 128 && masked) sum = capped_weights<KT, true>(s, ops, base, first, last, col_s);
        else sum = capped_weights<KT, false>(s, ops, base, first, last, col_s);
      } else {
        sum = weights<KT, MOD == 0>(s, ops.c2, base, col_s);
      }
      l += sum;
      if (dead) {
        if (!mbar_wait(kv_full + st, (n / NST) & 1, wc)) ok = false;   // landed before the scores were computed
        Tile::zero_row(sv + st * Cfg::KV_B, tid, KT);
        fence_proxy_async_smem();
      }
      __syncwarp();
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_warp(p_full + w);
    }
    if (n_w > 0 && ok) ok = mbar_wait_warp(o_full + w, 0, wc);
    // a cluster's partial results go over the operands: no product may still read those
    const bool in_cluster = p.splits > 1 && p.splits <= kAttnClusterSplits;
    if (in_cluster && ntiles > 0) ok = mbar_wait_warp(all_done, 0, wc) && ok;
    ok = __all_sync(~0u, ok);
    if (q0 + w * QT + wq * 32 < p.mask.Nq) {
      tc_fence_after();
      const bool have = row < p.mask.Nq;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const float lse2 = l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;   // l: NaN
      const long at = (static_cast<long>(b) * p.Hq + h) * p.mask.Nq + row;
      const long part_row = static_cast<long>(split) * BH * p.mask.Nq + at;
      if (in_cluster) {
        reinterpret_cast<float*>(sm + Cfg::OFF_LSE)[w * QT + tid] = lse2;
      } else if (have && ok) {
        if (p.splits > 1) p.part_l[part_row] = lse2;
        else if (p.L) p.L[at] = natural_lse(p, mask, h, row, lse2);
      }
      uint16_t* y = p.y + b * p.ys[0] + h * p.ys[1] + static_cast<long>(row) * p.ys[2];
#pragma unroll
      for (int d = 0; d < D; d += 16) {
        uint32_t o[16];
        if (n_w > 0) {
          tmem_ld16(col_o + d, o);
          tmem_wait_ld();
          regs_loaded(o);
        }
        float v[16];
        const bool zero = n_w == 0 || l == 0.f;   // a row that saw no key: whatever O holds
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = zero ? 0.f : __uint_as_float(o[i]) * (l > 0.f ? inv : l);
        if (in_cluster || (have && ok && p.splits > 1)) {
          float4* dst = reinterpret_cast<float4*>(in_cluster ? reinterpret_cast<float*>(sm) + (w * QT + tid) * Cfg::PART + d
                                                             : p.part_o + part_row * D + d);
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else if (have && ok) {
          uint4* dst = reinterpret_cast<uint4*>(y + d);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            dst[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
        }
      }
    }
  }
  // TMEM is given back before the CTA waits for the others of its cluster: one
  // that has not begun may be waiting for columns that depend on these
  tc_fence_before();
  __syncthreads();
  if (warp == Cfg::MMAS) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::TMEM_COLS);
  }
  if (p.splits > 1 && p.splits <= kAttnClusterSplits) {
    __syncwarp();
    cluster_sync();
    if (warp < 4 * NQ)
      cluster_join<D, Cfg::PART>(p.splits, split, reinterpret_cast<float*>(sm), reinterpret_cast<float*>(sm + Cfg::OFF_LSE),
                                 min(NQ * QT, p.mask.Nq - q0), threadIdx.x, 128 * NQ, [&](int r, int d, float4 v, float lse2) {
                                   const int row = q0 + r;
                                   *reinterpret_cast<uint2*>(p.y + b * p.ys[0] + h * p.ys[1] + static_cast<long>(row) * p.ys[2] + d) =
                                       make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                                   if (d == 0 && p.L)
                                     p.L[(static_cast<long>(b) * p.Hq + h) * p.mask.Nq + row] = natural_lse(p, mask, h, row, lse2);
                                 });
    __syncwarp();
    cluster_sync();   // the others have read this CTA's rows
  }
  if (warp == Cfg::LOADS && lane == 0 && ntiles > 0) {   // copies still in flight (only after an abort) must land before exit
    for (int st = 0; st < NST; ++st)
      if (last_load[st] >= 0) mbar_wait_drain(kv_full + st, (last_load[st] / NST) & 1, p.timeout_ns);
    for (int w = 0; w < NQ; ++w) mbar_wait_drain(q_full + w, 0, p.timeout_ns);
  }
}

// Join of the splits of one row: weights 2^(l_s - max).  Eight warps take the
// splits in turn (one warp's loads would wait for one another: 13 splits of 512
// rows 7 us, so 5).
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnParams p) {
  constexpr int WARPS = 8;
  __shared__ float part[WARPS][129];
  const long rows = static_cast<long>(p.B) * p.Hq * p.mask.Nq, at = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float top = -INFINITY;
  for (int s = lane; s < p.splits; s += 32) top = fmaxf(top, p.part_l[s * rows + at]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  const float base = top == -INFINITY ? 0.f : top;
  float total = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = warp; s < p.splits; s += WARPS) {
    const float w = ex2_mufu(p.part_l[s * rows + at] - base);
    total += w;
    const float* o = p.part_o + (s * rows + at) * p.D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < p.D) acc[i] = fmaf(w, o[lane + 32 * i], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[warp][lane + 32 * i] = acc[i];
  if (lane == 0) part[warp][128] = total;
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= p.D) return;
  float x = 0.f;
  total = 0.f;
#pragma unroll
  for (int k = 0; k < WARPS; ++k) {
    total += part[k][128];
    x += part[k][d];
  }
  const int n = static_cast<int>(at % p.mask.Nq);
  const long bh = at / p.mask.Nq;
  const int b = static_cast<int>(bh / p.Hq), h = static_cast<int>(bh % p.Hq);
  p.y[b * p.ys[0] + h * p.ys[1] + n * p.ys[2] + d] =
      static_cast<uint16_t>(pack_bf16x2(total == 0.f ? 0.f : x * (1.f / total), 0.f));
  if (d == 0 && p.L) p.L[at] = natural_lse(p, batch_mask(p.mask, b), h, n, total == 0.f ? -INFINITY : top + log2f(total));
}

// Documents: the start and the end of the run of equal ids each position lies
// in (the start twice where the id is negative).  A CTA takes 1024 positions:
// a bit for each that begins a run, then the nearest bit on either side.  Where
// runs reach into other chunks: with few chunks every CTA makes the bits of
// them all (ONE: one launch); with many a first launch (SUMS) leaves each
// chunk's last and first beginning in its first entry, a second turns them into
// what lies before and behind each chunk, a third (ENDS) does the rest.
// Latency: 8192 keys 4 us, 32768 8, 2^20 20.
constexpr int kDocThreads = 1024, kDocChunk = 1024, kDocOne = 16;   // chunks done in one launch
enum class Doc { ONE, SUMS, ENDS };
template <Doc HOW>
__global__ void __launch_bounds__(kDocThreads) attn_documents_kernel(const int32_t* ids, int2* doc, int N, int chunks) {
  constexpr int WORDS = kDocChunk / 32;
  __shared__ uint32_t all_bits[HOW == Doc::ONE ? kDocOne * WORDS : WORDS];
  __shared__ int left, right, before_word[WORDS], behind_word[WORDS];
  const int b = blockIdx.x / chunks, c0 = (blockIdx.x - b * chunks) * kDocChunk;
  const int from = HOW == Doc::ONE ? 0 : c0, words = HOW == Doc::ONE ? chunks * WORDS : WORDS;
  uint32_t* bits = all_bits + (c0 - from) / 32;
  ids += static_cast<long>(b) * N;
  doc += static_cast<long>(b) * N;
  const int t = threadIdx.x, lane = t & 31;
#pragma unroll 8
  for (int k = 0; k < 32 * words; k += kDocThreads) {
    const int i = from + k + t;
    const int id = i < N ? ids[i] : 0, edge = lane == 0 && i > 0 && i < N ? ids[i - 1] : 0;
    const int before = __shfl_up_sync(~0u, id, 1);
    const uint32_t w = __ballot_sync(~0u, i == 0 || i >= N || id != (lane == 0 ? edge : before));   // N begins what is behind
    if (lane == 0) all_bits[(k + t) / 32] = w;
  }
  if (threadIdx.x == 0) {
    left = HOW == Doc::ENDS ? doc[c0].x : -1;
    right = HOW == Doc::ENDS ? doc[c0].y : N;
  }
  __syncthreads();
  if constexpr (HOW != Doc::ENDS) {
    const int mine = (c0 - from) / 32;   // ONE: the words before and behind the chunk; SUMS: its own
    static_assert(kDocOne * WORDS <= kDocThreads, "a thread a word");
    if (t < words && all_bits[t]) {
      if (HOW == Doc::SUMS || t < mine) atomicMax(&left, from + 32 * t + 31 - __clz(all_bits[t]));
      if (HOW == Doc::SUMS || t >= mine + WORDS) atomicMin(&right, from + 32 * t + __ffs(all_bits[t]) - 1);
    }
    __syncthreads();
    if (HOW == Doc::SUMS && t == 0) doc[c0] = make_int2(left, right);
  }
  if constexpr (HOW != Doc::SUMS) {
    static_assert(WORDS == 32, "a lane a word");
    if (t < WORDS) {   // the nearest beginnings before and behind each word
      int x = bits[t] ? c0 + 32 * t + 31 - __clz(bits[t]) : -1, y = bits[t] ? c0 + 32 * t + __ffs(bits[t]) - 1 : N;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int a = __shfl_up_sync(~0u, x, o), z = __shfl_down_sync(~0u, y, o);
        if (t >= o) x = max(x, a);
        if (t + o < 32) y = min(y, z);
      }
      x = __shfl_up_sync(~0u, x, 1);
      y = __shfl_down_sync(~0u, y, 1);
      before_word[t] = t > 0 ? max(x, left) : left;
      behind_word[t] = t < 31 ? min(y, right) : right;
    }
    __syncthreads();
#pragma unroll
    for (int k = t; k < kDocChunk; k += kDocThreads) {
      const int i = c0 + k, w = k / 32;
      if (i >= N) break;
      const uint32_t m = bits[w] & (~0u >> (31 - lane)), z = lane == 31 ? 0u : bits[w] & (~0u << (lane + 1));
      const int start = m ? c0 + 32 * w + 31 - __clz(m) : before_word[w];
      const int end = z ? min(c0 + 32 * w + __ffs(z) - 1, N) : behind_word[w];
      doc[i] = make_int2(start, ids[i] < 0 ? start : end);
    }
  }
}

// A batch's chunks: (last, first beginning in the chunk) to (last beginning
// before it, first one behind it).  One CTA, a range of chunks per thread.
constexpr int kDocJoin = 1024;
__global__ void __launch_bounds__(kDocJoin) attn_document_ends_kernel(int2* doc, int N, int chunks) {
  __shared__ int last[kDocJoin], first[kDocJoin];
  const int t = threadIdx.x, per = (chunks + kDocJoin - 1) / kDocJoin;
  doc += static_cast<long>(blockIdx.x) * N;
  const int beg = min(chunks, t * per), end = min(chunks, beg + per);
  auto at = [&](int c) -> int2& { return doc[static_cast<long>(c) * kDocChunk]; };
  int x = -1, y = N;
  for (int c = beg; c < end; ++c) {
    x = max(x, at(c).x);
    y = min(y, at(c).y);
  }
  last[t] = x;
  first[t] = y;
  __syncthreads();
  for (int o = 1; o < kDocJoin; o *= 2) {   // inclusive, from the left and from the right
    const int a = t >= o ? last[t - o] : -1, z = t + o < kDocJoin ? first[t + o] : N;
    __syncthreads();
    last[t] = max(last[t], a);
    first[t] = min(first[t], z);
    __syncthreads();
  }
  x = t > 0 ? last[t - 1] : -1;
  y = t + 1 < kDocJoin ? first[t + 1] : N;
  for (int c = beg; c < end; ++c) {
    const int here = at(c).x;
    at(c).x = x;
    x = max(x, here);
  }
  for (int c = end - 1; c >= beg; --c) {
    const int here = at(c).y;
    at(c).y = y;
    y = min(y, here);
  }
}

}  // namespace

cudaError_t launch_attn_documents(const int32_t* ids, int2* doc, int B, int N, cudaStream_t s) {
  const int chunks = (N + kDocChunk - 1) / kDocChunk;
  const unsigned grid = static_cast<unsigned>(static_cast<long>(B) * chunks);
  if (chunks <= kDocOne) {
    attn_documents_kernel<Doc::ONE><<<grid, kDocThreads, 0, s>>>(ids, doc, N, chunks);
  } else {
    attn_documents_kernel<Doc::SUMS><<<grid, kDocThreads, 0, s>>>(ids, doc, N, chunks);
    attn_document_ends_kernel<<<static_cast<unsigned>(B), kDocJoin, 0, s>>>(doc, N, chunks);
    attn_documents_kernel<Doc::ENDS><<<grid, kDocThreads, 0, s>>>(ids, doc, N, chunks);
  }
  return cudaGetLastError();
}

namespace {
// Calls f with the kernel's configuration for these scores.
template <typename F>
auto by_config(const int D, bool bias, bool cap, F&& f) {
  auto by_mod = [&](auto d) {
    constexpr int DD = decltype(d)::value;
    return bias  ? f(d, std::integral_constant<int, 2>{}, FwdCfg<DD, 2>{})
           : cap ? f(d, std::integral_constant<int, 1>{}, FwdCfg<DD, 1>{})
                 : f(d, std::integral_constant<int, 0>{}, FwdCfg<DD, 0>{});
  };
  return D == 16   ? by_mod(std::integral_constant<int, 16>{})
         : D == 32 ? by_mod(std::integral_constant<int, 32>{})
         : D == 64 ? by_mod(std::integral_constant<int, 64>{})
                   : by_mod(std::integral_constant<int, 128>{});
}
}  // namespace

int attn_fwd_key_tile(int D, bool bias, bool cap) {
  return by_config(D, bias, cap, [](auto, auto, auto c) { return decltype(c)::KT; });
}

cudaError_t launch_attn_fwd(const AttnMaps& m, const AttnParams& p, cudaStream_t s) {
  return by_config(p.D, p.slopes != nullptr, p.cap > 0.f, [&](auto d, auto mod, auto c) {
    using C = decltype(c);
    const long n_qt = (p.mask.Nq + C::NQ * kAttnQTile - 1) / (C::NQ * kAttnQTile);
    const dim3 grid(static_cast<unsigned>(n_qt * p.B * p.Hq), static_cast<unsigned>(p.splits));
    auto* kern = attn_fwd_kernel<decltype(d)::value, decltype(mod)::value>;
    // at most CTAS CTAs share an SM, so that each finds its TMEM columns free
    constexpr int floor = 228 * 1024 / (C::CTAS + 1) + 1024;
    constexpr int smem = C::BYTES + 1024 > floor ? C::BYTES + 1024 : floor;
    const cudaError_t e = allow_smem<std::pair<C, decltype(mod)>>(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_splits(kern, grid, C::THREADS, smem, s, dim3(1, p.splits, 1), p.splits, m.q, m.k, m.v, p);
  });
}

cudaError_t launch_attn_join(const AttnParams& p, cudaStream_t s) {
  const long rows = static_cast<long>(p.B) * p.Hq * p.mask.Nq;
  attn_join_kernel<<<static_cast<unsigned>(rows), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace flare
