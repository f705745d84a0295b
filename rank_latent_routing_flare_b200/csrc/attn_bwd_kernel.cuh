// Exact softmax attention, backward, on tcgen05.  With P = 2^(x - l2) from the
// forward's row sums, g = <dY_i, v_j>, delta_i = <dY_i, Y_i> and x' the
// derivative of the capped score (1 without a cap):
//
//   dV_j = sum_i P_ij dY_i      dS_ij = P_ij (g_ij - delta_i) x'_ij
//   dQ_i = scale sum_j dS_ij k_j     dK_j = scale sum_i dS_ij q_i
//
// One kernel, two passes, so that every output is summed in one accumulator
// in a fixed order (no atomics).  A CTA keeps a tile of 128 rows and streams
// tiles of T rows of the other side:
//
//   dQ pass  rows: queries (Q, dY), stream: keys (K, V)
//     S = Q K^T, G = dY V^T, out1 += dS K, dS as two bf16 parts
//   dK/dV pass  rows: keys (K, V), stream: the rows (Q, dY) of every query
//     head of the key head, S = K Q^T, G = V dY^T, out1 += dS Q, out2 += P dY
//
// The rows are TMEM lanes (UMMA M = 128).  There are two pairs of S and G
// columns.  Weights and dS are written over S and G as bf16 and read from there
// as the products' A operands; the MMA warp issues tile n's products and right
// behind them the scores of tile n + 2 into the same columns (the tensor pipe
// runs in order), while the softmax threads work on tile n + 1.  D >= 64: four
// warpgroups share a tile, a quarter of its columns each, so that its weights
// are ready before the tensor pipe runs dry.  D <= 32: two take tiles in turn.
// Row statistics (l2, delta, interval) are held in registers in the dQ pass
// and come with the stream in the dK/dV pass.
//
// Roundings.  dS in bf16 is off by up to 2^-8 and would make dQ half again as
// inexact as its own rounding to bf16; the dQ pass, whose S columns are free,
// keeps dS - bf16(dS) there and adds its product too.  delta from the rounded
// Y would do the same where a row sees few keys: the dQ pass sums delta
// = sum_j P_ij g_ij in fp32 on the way and leaves it for the dK/dV pass, and with
// few keys it sums in a first sweep over them and has the use of it itself.  L in
// fp32 is coarse for a row far from its keys under a distance bias: there the
// dQ pass also sums P, which should be 1, divides by it and corrects l2 for the
// other pass.
//
// Few key heads under many rows leave most SMs without a tile in the dK/dV
// pass: there up to eight CTAs, a cluster, share a tile's stream and add their
// partial sums in a fixed order over each other's shared memory.
//
// Streamed rows that take no part (padding; in the dQ pass every key that no
// row of the tile sees) are zeroed in shared memory before the products read
// them: a weight of 0 does not erase a NaN.
//
// D >= 64: T = 64, up to 512 TMEM columns, one CTA per SM.  D <= 32: T = 48, 256
// columns, two CTAs per SM; the exponentials bound those.  Measured, dQ and
// dK/dV pass: D = 128, 2 x 16 heads (4 key heads) x 4095^2, capped, causal with
// prefixes 324 and 312 us (0.94 PFLOP/s over their four products each); D = 32,
// 8 x 8 heads x 4096^2, ragged, 222 and 294.
#pragma once

#include <tuple>
#include <type_traits>
#include <utility>

#include "attn_common.cuh"
#include "ops_internal.h"

namespace flare {

// Up to this many keys the dQ pass sums delta and the weights before it uses
// them: delta from the rounded Y is off by what one key weighs.  Norm of dQ's
// error, of its values' rounding to bf16, with one sweep (two): 1.4 (1.0) at 100
// keys, 1.2 (1.0) at 370, 1.5 (1.0) at 900 under a bias, 1.15 at 2000, 1.1 at
// 4000.  The first sweep adds 40 to 90 % to this pass, at such sizes 3 to 6 us
// of a step that takes 50 to 60 on the host; at 4000 keys it would be a quarter of the step.
constexpr int kAttnTwiceKeys = 1024;

template <int D_, bool KV>
struct BwdCfg {
  static constexpr int D = D_;
  using Tile = RowTile<D>;
  static constexpr int T = D <= 32 ? 48 : 64;
  // Wide heads, one CTA an SM: four warpgroups share a tile, a quarter of its
  // columns each.  Narrow ones, two CTAs an SM: two warpgroups take tiles in turn.
  static constexpr bool SHARE = D >= 64;
  static constexpr int CTAS = SHARE ? 1 : 2, WGS = SHARE ? 4 : 2;
  static constexpr int COLS = SHARE ? T / WGS : T;        // columns of a tile per warpgroup
  static constexpr int CH = 16 < COLS ? 16 : COLS;        // columns computed at once
  static constexpr int OUTS = KV ? 2 : 1;
  // Rows kept in TMEM, as the A operands of the score products, where columns
  // are left: from shared memory an A operand of 128 rows takes as long to read
  // as the product of 64 columns.
  static constexpr bool XT = D >= 64 && 4 * T + (OUTS + 1) * D <= 512;
  static constexpr int NST = D == 128 ? (XT ? 384 : 256) / T : 6;
  static constexpr int X_B = XT ? 0 : Tile::bytes(128), Y_B = Tile::bytes(T), R_B = kAttnRowFields * T * 4;
  static constexpr int OFF_X = 0;                         // X1 | X2
  static constexpr int OFF_Y = OFF_X + 2 * X_B;           // NST x (Y1 | Y2)
  static constexpr int OFF_R = OFF_Y + 2 * NST * Y_B;     // NST x row statistics (dK/dV pass); sums of the warpgroups (dQ pass)
  static constexpr int OFF_BAR = OFF_R + (KV ? NST * R_B : WGS * 1024);
  static constexpr int OFF_MISC = OFF_BAR + 8 * (1 + 2 * NST + 2 + 2 + 1);
  static constexpr int BYTES = OFF_MISC + 32 + 4 * NST;
  // buffer g: S at 2 T g, G at 2 T g + T
  static constexpr uint32_t COL_S = 0, COL_OUT1 = 4 * T, COL_OUT2 = 4 * T + D, COL_X1 = 4 * T + OUTS * D, COL_X2 = COL_X1 + D / 2;
  static constexpr uint32_t COL_END = XT ? COL_X2 + D / 2 : COL_X1;
  static constexpr uint32_t TMEM_COLS = COL_END <= 256 ? 256 : 512;
  static constexpr int LOADS = 4 * WGS, MMAS = 4 * WGS + 1, THREADS = 32 * (4 * WGS + 2);   // warps: softmax, loads, MMAs
  static_assert(COL_END <= TMEM_COLS && TMEM_COLS * CTAS <= 512, "TMEM columns");
  static_assert(COLS % 16 == 0 && Y_B % (8 * Tile::ROWB) == 0 && X_B % 1024 == 0 && R_B % 64 == 0, "tiles hold whole swizzle atoms");
  static constexpr int PART = OUTS * D + 4;               // floats between rows of a split's partial outputs
  static_assert(!KV || 128 * PART * 4 <= OFF_BAR, "partial outputs go over the operands and the statistics");
  static_assert(BYTES + 1024 <= 227 * 1024, "shared memory");
};

// MOD: 0 plain scores, 1 capped, 2 with a distance bias (and capped if p.cap > 0).
// TWICE (dQ pass): a first sweep over the keys sums delta and the weights.
template <int D, bool KV, int MOD, bool TWICE>
__global__ void __launch_bounds__(BwdCfg<D, KV>::THREADS, BwdCfg<D, KV>::CTAS)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_x1, const __grid_constant__ CUtensorMap tm_x2,
                    const __grid_constant__ CUtensorMap tm_y1, const __grid_constant__ CUtensorMap tm_y2,
                    const AttnBwdParams bp) {
  using Cfg = BwdCfg<D, KV>;
  using Tile = RowTile<D>;
  constexpr int T = Cfg::T, NST = Cfg::NST, CH = Cfg::CH, TR = BwdCfg<D, true>::T;   // TR: rows of a block of statistics
  const AttnParams& p = bp.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sx = sm + Cfg::OFF_X;
  uint8_t* sy = sm + Cfg::OFF_Y;
  uint8_t* sr = sm + Cfg::OFF_R;
  uint64_t* x_full = reinterpret_cast<uint64_t*>(sm + Cfg::OFF_BAR);
  uint64_t* y_full = x_full + 1;          // [NST]
  uint64_t* y_empty = y_full + NST;       // [NST] products of the tile done
  uint64_t* s_full = y_empty + NST;       // [2] scores and G of the warpgroup's next tile ready
  uint64_t* p_full = s_full + 2;          // [2] weights and dS stored (one arrive per warp)
  uint64_t* all_done = p_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Cfg::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(sm + Cfg::OFF_MISC + 4);
  volatile int* range = reinterpret_cast<volatile int*>(sm + Cfg::OFF_MISC + 8);       // [6]
  volatile int* last_load = reinterpret_cast<volatile int*>(sm + Cfg::OFF_MISC + 32);  // [NST]

  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // the dQ pass owns query heads and begins with the last rows, the dK/dV
  // pass owns key heads and begins with the first keys: under a causal mask
  // those have the most to do
  const int split_bits = KV ? bp.split_bits : 0, splits = 1 << split_bits, split = blockIdx.x & (splits - 1);
  const int block = static_cast<int>(blockIdx.x) >> split_bits, blocks = static_cast<int>(gridDim.x) >> split_bits;
  const int heads = KV ? p.Hk : p.Hq, n_tiles = blocks / (p.B * heads);
  const int ti = block / (p.B * heads), bh = block % (p.B * heads);
  const int x0 = (KV ? ti : n_tiles - 1 - ti) * 128;
  const int b = bh / heads, hx = bh % heads;
  const BatchMask mask = batch_mask(p.mask, b);

  // Stream tiles [range0, range1) that take part, and of the stream's rows those
  // [range2, range3) that every row of this tile that takes part sees (dQ
  // pass), or that see all of its keys.  dQ pass: the first and the last key
  // that one of them sees, [range4, range5).
  if (threadIdx.x < (KV ? 4 : 6)) {
    const int what = threadIdx.x;
    int v = 0;
    if (KV) {   // hi > x0 from the first row on, lo < x0 + 128 up to the last; hi >= x0 + 128, lo <= x0
      int lo = 0, hi = mask.qlen;
      while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        const int2 iv = row_interval(mask, mid);
        const bool behind = what == 0 ? iv.y > x0 : what == 1 ? iv.x >= x0 + 128 : what == 2 ? iv.y >= x0 + 128 : iv.x > x0;
        if (behind) hi = mid; else lo = mid + 1;
      }
      v = what == 0 ? lo / T : what == 1 ? (lo + T - 1) / T : lo;
    } else {
      const int r1 = min(x0 + 128, mask.qlen);
      if (x0 < r1) {
        const int2 a = row_interval(mask, x0), z = row_interval(mask, r1 - 1);
        if (a.x < z.y)
          v = what == 0 ? a.x / T : what == 1 ? (z.y + T - 1) / T : what == 2 ? z.x : what == 3 ? a.y : what == 4 ? a.x : z.y;
      }
    }
    range[what] = v;
  }
  if (threadIdx.x == 64) {
    mbar_init(x_full, Cfg::XT ? 4 * Cfg::WGS : 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, Cfg::SHARE ? 4 * Cfg::WGS : 4);
    }
    for (int i = 0; i < NST; ++i) {
      mbar_init(y_full + i, 1);
      mbar_init(y_empty + i, 1);
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
  const int t_lo = range[0], per_head = max(0, range[1] - range[0]), whole0 = range[2], whole1 = range[3];
  // stream tiles: the split's share of those of all heads, one head's behind the other's
  const long all = static_cast<long>(per_head) * (KV ? p.G : 1);
  const int n0 = static_cast<int>(all * split >> split_bits), N1 = static_cast<int>(all * (split + 1) >> split_bits) - n0;
  const int N0 = TWICE ? N1 : 0;                  // steps that only sum
  const int N = N0 + N1;

  if (warp >= Cfg::LOADS) {
    if (warp == Cfg::LOADS) {
      // ------------------------------------------------------------ loads
      if (lane == 0 && N > 0) {
        if (!Cfg::XT) {
          tma_prefetch_desc(&tm_x1);
          tma_prefetch_desc(&tm_x2);
        }
        tma_prefetch_desc(&tm_y1);
        tma_prefetch_desc(&tm_y2);
        if (!Cfg::XT) {
          mbar_arrive_expect_tx(x_full, 2 * Cfg::X_B);
          Tile::load(sx, &tm_x1, x_full, x0, hx, b, 128);
          Tile::load(sx + Cfg::X_B, &tm_x2, x_full, x0, hx, b, 128);
        }
        for (int n = 0; n < N; ++n) {
          const int st = n % NST;
          if (n >= NST && !mbar_wait(y_empty + st, (n / NST - 1) & 1, wc)) break;
          const int g = KV ? (n0 + n) / per_head : 0, row = (t_lo + (KV ? n0 + n - g * per_head : n < N0 ? n : n - N0)) * T;
          const int hy = KV ? hx * p.G + g : hx / p.G;
          mbar_arrive_expect_tx(y_full + st, 2 * Cfg::Y_B + (KV ? Cfg::R_B : 0));
          Tile::load(sy + 2 * st * Cfg::Y_B, &tm_y1, y_full + st, row, hy, b, T);
          Tile::load(sy + (2 * st + 1) * Cfg::Y_B, &tm_y2, y_full + st, row, hy, b, T);
          if (KV)
            bulk_load(sr + st * Cfg::R_B, bp.rows + ((static_cast<long>(b) * p.Hq + hy) * bp.row_blocks + row / T) *
                      (kAttnRowFields * T), Cfg::R_B, y_full + st);
          last_load[st] = n;
        }
      }
    } else {
      // ------------------------------------------------------------ MMAs
      if (N > 0) {   // the whole warp, converged
        const uint32_t idesc_s = idesc_bf16_f32(128, T, false, false);
        const uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
        const uint64_t x1 = Tile::desc_k(sx), x2 = Tile::desc_k(sx + Cfg::X_B);
        const uint64_t y_k = Tile::desc_k(sy), y_mn = Tile::desc_mn(sy, T);
        constexpr uint64_t TILE = Cfg::Y_B >> 4;
        // columns of a k-step of 16 weights: each warpgroup packs its own into the first half of its columns
        auto a_col = [](int ks) { return 16 * ks / Cfg::COLS * Cfg::COLS + 16 * ks % Cfg::COLS / 2; };
        auto landed = [&](int n) { return n >= N || mbar_wait_warp(y_full + n % NST, (n / NST) & 1, wc); };
        auto issue_scores = [&](int n) {   // one lane
          const uint32_t col = tmem + Cfg::COL_S + (n & 1) * 2 * T;
          const uint64_t y1 = y_k + 2 * (n % NST) * TILE, y2 = y1 + TILE;
#pragma unroll
          for (int side = 0; side < 2; ++side)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t y = (side ? y2 : y1) + Tile::kstep_k(kk, T);
              if constexpr (Cfg::XT)
                umma_ts(col + side * T, tmem + (side ? Cfg::COL_X2 : Cfg::COL_X1) + 8 * kk, y, idesc_s, kk > 0 ? 1u : 0u);
              else
                umma_ss(col + side * T, (side ? x2 : x1) + Tile::kstep_k(kk, 128), y, idesc_s, kk > 0 ? 1u : 0u);
            }
          umma_commit(s_full + (n & 1));
        };
        bool ok = mbar_wait_warp(x_full, 0, wc) && landed(0) && landed(1);
        tc_fence_after();
        if (ok && elect_one()) {
          issue_scores(0);
          if (N > 1) issue_scores(1);
        }
        __syncwarp();
        for (int n = 0; ok && n < N; ++n) {
          // the scores of tile n + 2 follow the products of tile n without a gap
          ok = landed(n + 2) && mbar_wait_warp(p_full + (n & 1), (n >> 1) & 1, wc);
          if (!ok) break;
          tc_fence_after();
          const int st = n % NST;
          const uint32_t col = tmem + Cfg::COL_S + (n & 1) * 2 * T;
          const uint64_t y1 = y_mn + 2 * st * TILE, y2 = y1 + TILE;
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < T / 16; ++ks)
              if (n >= N0)
                umma_ts(tmem + Cfg::COL_OUT1, col + T + a_col(ks), y1 + ks * Tile::KSTEP_MN, idesc_o, (n > N0 || ks > 0) ? 1u : 0u);
#pragma unroll
            for (int ks = 0; ks < T / 16; ++ks) {
              if (KV)
                umma_ts(tmem + Cfg::COL_OUT2, col + a_col(ks), y2 + ks * Tile::KSTEP_MN, idesc_o, (n > 0 || ks > 0) ? 1u : 0u);
              else if (n >= N0)   // the low parts of dS
                umma_ts(tmem + Cfg::COL_OUT1, col + a_col(ks), y1 + ks * Tile::KSTEP_MN, idesc_o, 1u);
            }
            umma_commit(y_empty + st);
            if (n + 2 < N) issue_scores(n + 2);
          }
          __syncwarp();
        }
        if (elect_one()) umma_commit(all_done);
        __syncwarp();
        mbar_wait_drain(all_done, 0, p.timeout_ns);
        __syncwarp();
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int w = warp >> 2, wq = warp & 3;
    const int tid = threadIdx.x & 127;
    const int row = x0 + tid;                       // query (dQ pass) or key of this lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    constexpr int COLS = Cfg::COLS;
    const int c0 = Cfg::SHARE ? w * COLS : 0;      // this warpgroup's columns of a tile
    const ScoreOps ops(p.scale, p.cap, false);
    const bool capped = MOD == 1 || (MOD == 2 && p.cap > 0.f);
    // dQ pass: this row's statistics
    float nl2 = -INFINITY, ndelta = 0.f, slope2 = 0.f;
    int lo = 0, hi = 0, pos = 0;
    float* stat = bp.rows + ((static_cast<long>(b) * p.Hq + hx) * bp.row_blocks + row / TR) * (kAttnRowFields * TR) + row % TR;
    if (!KV) {
      if (row < p.mask.Nq) {
        nl2 = stat[0];
        ndelta = stat[TR];
        lo = __float_as_int(stat[2 * TR]);
        hi = __float_as_int(stat[3 * TR]);
        pos = __float_as_int(stat[4 * TR]);
      }
      if (MOD == 2) slope2 = p.slopes[hx] * kLog2e;
    }
    constexpr bool SUM_P = !KV && (MOD == 2 || TWICE);
    uint64_t delta2 = f2_dup(0.f), total2 = delta2;  // dQ pass: sums of P g and (SUM_P) of P
    bool ok = true;
    if (Cfg::XT && N > 0) {   // this lane's row of X1 (the first half of the warpgroups) or X2 into TMEM
      constexpr int EACH = 2 * D / Cfg::WGS;          // elements a warpgroup brings
      const bool first = w < Cfg::WGS / 2;
      const int d0 = w % (Cfg::WGS / 2) * EACH;
      const AttnSide& src = KV ? (first ? bp.k : bp.v) : (first ? bp.q : bp.dy);
      const uint16_t* xr = src.p + b * src.sb + hx * src.sh + static_cast<long>(row) * src.sn + d0;
      const bool have = row < (KV ? p.mask.Nk : p.mask.Nq);
#pragma unroll
      for (int d = 0; d < EACH; d += 32) {
        uint32_t r[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = have ? *reinterpret_cast<const uint4*>(xr + d + 8 * i) : make_uint4(0, 0, 0, 0);
          r[4 * i] = v.x;
          r[4 * i + 1] = v.y;
          r[4 * i + 2] = v.z;
          r[4 * i + 3] = v.w;
        }
        tmem_st16(lane_base + (first ? Cfg::COL_X1 : Cfg::COL_X2) + (d0 + d) / 2, r);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_warp(x_full);
    }
    // query head of the key head, tile of that head's stream
    int g = KV && n0 > 0 ? n0 / per_head : 0, tn = n0 - g * per_head + (Cfg::SHARE ? 0 : w);
    // dQ pass, once per thread: the warpgroups' sums, and delta and l2 as they
    // come out, for the dK/dV pass
    float inv_total = 1.f;
    auto settle = [&] {
      float d0, d1, t0, t1;
      f2_unpack(delta2, d0, d1);
      f2_unpack(total2, t0, t1);
      float2* share = reinterpret_cast<float2*>(sr);
      share[w * 128 + tid] = make_float2(d0 + d1, t0 + t1);
      named_bar_sync(1, 128 * Cfg::WGS);
      float2 a = share[tid];
#pragma unroll
      for (int i = 1; i < Cfg::WGS; ++i) {
        const float2 c = share[128 * i + tid];
        a.x += c.x;
        a.y += c.y;
      }
      const float total = SUM_P ? a.y : 1.f;
      inv_total = total > 0.f ? 1.f / total : total;   // NaN stays
      if (nl2 != -INFINITY) {
        ndelta = -a.x * inv_total;
        if (w == 0 && row < p.mask.Nq) {
          stat[0] = nl2 - log2f(total);
          stat[TR] = ndelta;
        }
      }
    };
    bool settled = KV;
    for (int n = Cfg::SHARE ? 0 : w; n < N; n += Cfg::SHARE ? 1 : 2, tn += Cfg::SHARE ? 1 : 2) {
      if (KV)
        for (; tn >= per_head; tn -= per_head) ++g;
      if (TWICE && !settled && n >= N0) {
        settle();
        settled = true;
        tn -= N0;
      }
      const int st = n % NST, buf = n & 1;
      const uint32_t col_s = lane_base + Cfg::COL_S + buf * 2 * T + c0, col_g = col_s + T;
      const int y0 = (t_lo + tn) * T;
      if (KV && MOD == 2) slope2 = p.slopes[hx * p.G + g] * kLog2e;
      const float* rs = reinterpret_cast<const float*>(sr + st * Cfg::R_B);
      const int* ri = reinterpret_cast<const int*>(rs);
      // the statistics come with the tile; waiting for it makes them visible to this thread
      if (KV && !mbar_wait_warp(y_full + st, (n / NST) & 1, wc)) { ok = false; break; }
      const bool full = y0 >= whole0 && y0 + T <= whole1;
      bool dead = false;                            // the streamed row this thread answers for takes no part
      if (!full && tid < T && (!Cfg::SHARE || w == 0)) {
        if (KV) {
          dead = rs[tid] == -INFINITY;
        } else if (y0 + tid < mask.nk) {
          dead = y0 + tid < range[4] || y0 + tid >= range[5];
          if (mask.doc) {
            const int2 d = mask.doc[y0 + tid];
            dead |= d.x == d.y;
          }
        }
      }
      // dQ pass, bias: side 1 (-1) where every row of the warp stands behind (before) all keys of the tile
      const int side = KV || MOD != 2 ? 0 : __all_sync(~0u, pos >= y0 + T - 1) ? 1 : __all_sync(~0u, pos <= y0) ? -1 : 0;
      if (!mbar_wait_warp(s_full + buf, (n >> 1) & 1, wc)) { ok = false; break; }
      tc_fence_after();
      // one body for tiles that every row sees whole, one for the others
      auto tile = [&](auto whole) {
        constexpr bool FULL = decltype(whole)::value;
        constexpr bool AHEAD = MOD != 2;            // the next columns' read in flight; the bias needs those registers
        uint32_t s[2][CH], gg[2][CH];
        tmem_ld_cols<CH>(col_s, s[0]);
        tmem_ld_cols<CH>(col_g, gg[0]);
        tmem_wait_ld();
        regs_loaded(s[0]);
        regs_loaded(gg[0]);
#pragma unroll
        for (int c = 0; c < COLS; c += CH) {
          constexpr int NB = CH;
          const int cur = (c / CH) & 1;
          if (AHEAD && c + CH < COLS) {
            tmem_ld_cols<NB>(col_s + c + CH, s[cur ^ 1]);
            tmem_ld_cols<NB>(col_g + c + CH, gg[cur ^ 1]);
          }
          uint32_t pk[CH / 2], dk[CH / 2], dl[CH / 2];
          const bool small = (MOD == 1 || capped) && MOD != 0 &&
                             __all_sync(~0u, ops.small(fmaxf(max_of(s[cur]), -min_of(s[cur]))));
          // x - l2 of the columns, and 1 - tanh^2
          uint64_t x[CH / 2], dx[CH / 2];
#pragma unroll
          for (int q = 0; q < CH / 2; ++q) x[q] = f2(s[cur][2 * q], s[cur][2 * q + 1]);
          if (MOD == 1 || (MOD == 2 && capped)) {
            if (small) {
#pragma unroll
              for (int q = 0; q < CH / 2; ++q) x[q] = ops.poly(x[q], f2_dup(0.f));
            } else {
#pragma unroll
              for (int q = 0; q < CH / 2; ++q)
                x[q] = f2_pack(ops.tanh_any(as_f(s[cur][2 * q])), ops.tanh_any(as_f(s[cur][2 * q + 1])));
            }
#pragma unroll
            for (int q = 0; q < CH / 2; ++q) dx[q] = f2_fma(f2_mul(x[q], f2_dup(-1.f)), x[q], f2_dup(1.f));
          }
          const uint32_t bits = FULL || KV ? ~0u : column_bits(lo - y0 - c0, hi - y0 - c0, c);   // columns that the row sees
          const uint64_t f = f2_dup(capped ? ops.out : ops.c2);
          uint64_t b2 = f2_dup(0.f), step = b2;
          if (MOD == 2 && !KV && side != 0) step = f2_dup(side > 0 ? 2.f * slope2 : -2.f * slope2);
#pragma unroll
          for (int q = 0; q < CH / 2; q += 2) {
            float4 l4 = make_float4(nl2, nl2, nl2, nl2), d4 = make_float4(ndelta, ndelta, ndelta, ndelta);
            if (KV) {
              l4 = *reinterpret_cast<const float4*>(rs + c0 + c + 2 * q);
              d4 = *reinterpret_cast<const float4*>(rs + T + c0 + c + 2 * q);
            }
            const uint64_t ll[2] = {f2_pack(l4.x, l4.y), f2_pack(l4.z, l4.w)};
            const uint64_t dd[2] = {f2_pack(d4.x, d4.y), f2_pack(d4.z, d4.w)};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int k = c0 + c + 2 * (q + u);      // the pair's first column
              uint64_t t = f2_fma(x[q + u], f, ll[u]);
              if (MOD == 2) {
                if (KV) {
                  t = f2_add(t, f2_pack(-slope2 * fabsf(static_cast<float>(ri[4 * T + k] - row)),
                                        -slope2 * fabsf(static_cast<float>(ri[4 * T + k + 1] - row))));
                } else {
                  const float d = static_cast<float>(pos - y0);
                  if (side != 0) {
                    if ((q + u) % 8 == 0) {
                      const float gs = side > 0 ? -slope2 : slope2;
                      b2 = f2_pack(gs * (d - k), gs * (d - (k + 1)));
                    }
                    t = f2_add(t, b2);
                    b2 = f2_add(b2, step);
                  } else {
                    t = f2_add(t, f2_pack(-slope2 * fabsf(d - k), -slope2 * fabsf(d - (k + 1))));
                  }
                }
              }
              float p0, p1;
              ex2_pair(t, p0, p1);
              uint64_t pp = f2_pack(p0, p1);
              uint64_t pg = f2_mul(pp, f2(gg[cur][2 * (q + u)], gg[cur][2 * (q + u) + 1]));
              uint64_t ds = f2_fma(pp, dd[u], pg);     // P (g - delta)
              if (MOD == 1 || (MOD == 2 && capped)) ds = f2_mul(ds, dx[q + u]);
              if (!FULL) {
                float a0, a1, b0, b1;
                f2_unpack(ds, a0, a1);
                f2_unpack(pg, b0, b1);
                const bool h0 = KV ? row < ri[2 * T + k] || row >= ri[3 * T + k] : !(bits & (1u << (2 * (q + u))));
                const bool h1 = KV ? row < ri[2 * T + k + 1] || row >= ri[3 * T + k + 1] : !(bits & (2u << (2 * (q + u))));
                p0 = h0 ? 0.f : p0;
                p1 = h1 ? 0.f : p1;
                ds = f2_pack(h0 ? 0.f : a0, h1 ? 0.f : a1);
                pg = f2_pack(h0 ? 0.f : b0, h1 ? 0.f : b1);
              }
              float s0, s1;
              f2_unpack(ds, s0, s1);
              const uint32_t hi16 = pack_bf16x2(s0, s1);
              dk[q + u] = hi16;
              if (KV) {
                pk[q + u] = pack_bf16x2(p0, p1);
              } else {
                delta2 = f2_add(delta2, pg);
                if (SUM_P) total2 = f2_add(total2, f2_pack(p0, p1));
                f2_unpack(f2_fma(f2_pack(bf16_lo(hi16), bf16_hi(hi16)), f2_dup(-1.f), ds), s0, s1);
                dl[q + u] = pack_bf16x2(s0, s1);
              }
            }
          }
          tmem_st_cols<CH / 2>(col_s + c / 2, KV ? pk : dl);
          tmem_st_cols<CH / 2>(col_g + c / 2, dk);
          if (c + CH < COLS) {
            if (!AHEAD) {
              tmem_ld_cols<NB>(col_s + c + CH, s[cur ^ 1]);
              tmem_ld_cols<NB>(col_g + c + CH, gg[cur ^ 1]);
            }
            tmem_wait_ld();
            regs_loaded(s[cur ^ 1]);
            regs_loaded(gg[cur ^ 1]);
          }
        }
      };
      if (full) tile(std::true_type{});
      else tile(std::false_type{});
      if (dead) {
        if (!mbar_wait(y_full + st, (n / NST) & 1, wc)) ok = false;   // landed before the scores were computed
        Tile::zero_row(sy + 2 * st * Cfg::Y_B, tid, T);
        if (KV) Tile::zero_row(sy + (2 * st + 1) * Cfg::Y_B, tid, T);
        fence_proxy_async_smem();
      }
      __syncwarp();
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_warp(p_full + buf);
    }
    if (!settled) settle();                           // (TWICE: after an abort, or if the second sweep has no tile for it)
    if (ok && N > 0) ok = mbar_wait_warp(all_done, 0, wc);
    ok = __all_sync(~0u, ok);
    if (ok || splits > 1) {
      tc_fence_after();
      // the outputs' columns are dealt to the warpgroups, 16 at least each: dK then dV, or dQ
      constexpr int OUT = Cfg::OUTS * D, EACH = OUT / Cfg::WGS < 16 ? 16 : OUT / Cfg::WGS;
      const bool second = w * EACH >= D;
      const int d_beg = w * EACH - (second ? D : 0), d_end = w * EACH < OUT ? d_beg + EACH : d_beg;
      const uint32_t col = lane_base + (second ? Cfg::COL_OUT2 : Cfg::COL_OUT1);
      uint16_t* out = second ? bp.dv + b * bp.dvs[0] + hx * bp.dvs[1] + static_cast<long>(row) * bp.dvs[2]
                      : KV   ? bp.dk + b * bp.dks[0] + hx * bp.dks[1] + static_cast<long>(row) * bp.dks[2]
                             : bp.dq + b * bp.dqs[0] + hx * bp.dqs[1] + static_cast<long>(row) * bp.dqs[2];
      const float f = second ? 1.f : p.scale * inv_total;
      const bool have = row < (KV ? p.mask.Nk : p.mask.Nq);
      // a row that takes no part gets zeros, whatever its lane holds
      const bool zero = N == 0 || (KV ? row >= mask.len || (mask.doc && have && mask.doc[row].x == mask.doc[row].y)
                                      : nl2 == -INFINITY);
      for (int d = d_beg; d < d_end; d += 16) {
        uint32_t o[16];
        if (N > 0 && ok) {
          tmem_ld16(col + d, o);
          tmem_wait_ld();
          regs_loaded(o);
        }
        if (KV && splits > 1) {
          float4* part = reinterpret_cast<float4*>(reinterpret_cast<float*>(sm) + tid * Cfg::PART + (second ? D : 0) + d);
          const bool some = N > 0 && ok;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            part[i] = some ? make_float4(as_f(o[4 * i]), as_f(o[4 * i + 1]), as_f(o[4 * i + 2]), as_f(o[4 * i + 3]))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
          continue;
        }
        uint32_t pk[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          pk[i] = zero ? 0u : pack_bf16x2(__uint_as_float(o[2 * i]) * f, __uint_as_float(o[2 * i + 1]) * f);
        if (have) {
          uint4* dst = reinterpret_cast<uint4*>(out + d);
          dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
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
  __syncwarp();
  if (KV && splits > 1) {   // each CTA of the cluster adds up its share of the rows, in the splits' order
    cluster_sync();
    const int per = 128 / splits;
    for (int i = threadIdx.x; i < per * (2 * D / 8); i += Cfg::THREADS) {
      const int r = split * per + i / (2 * D / 8), c = 8 * (i % (2 * D / 8)), row = x0 + r;
      if (row >= p.mask.Nk) continue;
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
      const float* part = reinterpret_cast<const float*>(sm) + r * Cfg::PART + c;
      for (int k = 0; k < splits; ++k) {
        const float4 a = peer_load4(peer_smem(part, k)), e = peer_load4(peer_smem(part + 4, k));
        u = make_float4(u.x + a.x, u.y + a.y, u.z + a.z, u.w + a.w);
        v = make_float4(v.x + e.x, v.y + e.y, v.z + e.z, v.w + e.w);
      }
      const bool zero = all == 0 || row >= mask.len || (mask.doc && mask.doc[row].x == mask.doc[row].y);
      const float f = c >= D ? 1.f : p.scale;
      uint16_t* out = c >= D ? bp.dv + b * bp.dvs[0] + hx * bp.dvs[1] + static_cast<long>(row) * bp.dvs[2] + c - D
                             : bp.dk + b * bp.dks[0] + hx * bp.dks[1] + static_cast<long>(row) * bp.dks[2] + c;
      *reinterpret_cast<uint4*>(out) =
          zero ? make_uint4(0, 0, 0, 0) : make_uint4(pack_bf16x2(u.x * f, u.y * f), pack_bf16x2(u.z * f, u.w * f),
                                                     pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
    }
    cluster_sync();         // the others have read this CTA's rows
  }
  if (warp == Cfg::LOADS && lane == 0 && N > 0) {   // copies still in flight (only after an abort) must land before exit
    for (int st = 0; st < NST; ++st)
      if (last_load[st] >= 0) mbar_wait_drain(y_full + st, (last_load[st] / NST) & 1, p.timeout_ns);
    if (!Cfg::XT) mbar_wait_drain(x_full, 0, p.timeout_ns);
  }
}

// Splits of a key tile's stream in the dK/dV pass, as a power of two: as many
// as leave no CTA without an SM, with two tiles each or more.  Without (with)
// them, D = 128, causal: one key head of 8 query heads, 4096 rows, 477 us (135);
// D = 32: 8 heads of 64 keys under 8192 rows 150 us (30), 8 heads of 2000 rows
// 32 us (25).
inline int bwd_split_bits(long ctas, int per_sm, long stream) {
  int n = 0;
  while ((2 << n) <= kAttnClusterSplits && (ctas << (n + 1)) <= kNumSM * per_sm && (4 << n) <= stream) ++n;
  return n;
}

template <bool KV>
cudaError_t launch_attn_bwd_pass(const CUtensorMap& x1, const CUtensorMap& x2, const CUtensorMap& y1,
                                 const CUtensorMap& y2, const AttnBwdParams& p, cudaStream_t s) {
  const long tiles = ((KV ? p.a.mask.Nk : p.a.mask.Nq) + 127) / 128;
  const long ctas = tiles * p.a.B * (KV ? p.a.Hk : p.a.Hq);
  auto go = [&](auto d, auto mod, auto twice) {
    constexpr int D = decltype(d)::value;
    using C = BwdCfg<D, KV>;
    auto* kern = attn_bwd_kernel<D, KV, decltype(mod)::value, decltype(twice)::value>;
    // at most CTAS CTAs share an SM, so that each finds its TMEM columns free
    constexpr int floor = 228 * 1024 / (C::CTAS + 1) + 1024;
    constexpr int smem = C::BYTES + 1024 > floor ? C::BYTES + 1024 : floor;
    const cudaError_t e = allow_smem<std::tuple<C, decltype(mod), decltype(twice)>>(kern, smem);
    if (e != cudaSuccess) return e;
    AttnBwdParams q = p;
    q.split_bits = KV ? bwd_split_bits(ctas, C::CTAS, static_cast<long>(p.a.G) * ((p.a.mask.Nq + C::T - 1) / C::T)) : 0;
    return launch_splits(kern, dim3(static_cast<unsigned>(ctas << q.split_bits)), C::THREADS, smem, s,
                         dim3(1u << q.split_bits), 1 << q.split_bits, x1, x2, y1, y2, q);
  };
  auto by_sweeps = [&](auto d, auto mod) {
    if constexpr (!KV)
      if (p.a.mask.Nk <= kAttnTwiceKeys) return go(d, mod, std::true_type{});
    return go(d, mod, std::false_type{});
  };
  auto by_mod = [&](auto d) {
    return p.a.slopes      ? by_sweeps(d, std::integral_constant<int, 2>{})
           : p.a.cap > 0.f ? by_sweeps(d, std::integral_constant<int, 1>{})
                           : by_sweeps(d, std::integral_constant<int, 0>{});
  };
  switch (p.a.D) {
    case 16: return by_mod(std::integral_constant<int, 16>{});
    case 32: return by_mod(std::integral_constant<int, 32>{});
    case 64: return by_mod(std::integral_constant<int, 64>{});
    case 128: return by_mod(std::integral_constant<int, 128>{});
  }
  return cudaErrorInvalidValue;
}

}  // namespace flare
