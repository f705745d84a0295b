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
// no query may see (padding) are zeroed in shared memory by the softmax
// threads before the product.
//
// D = 128: KT = 128, 512 TMEM columns, one CTA per SM.  D <= 64: the
// exponentials bound the kernel; KT = 64 and 256 columns let two CTAs (four
// softmax warps per SM sub-partition) share an SM.
#include "attn_common.cuh"

namespace flare {
namespace {

template <int D>
struct FwdCfg {
  using Tile = RowTile<D>;
  static constexpr int KT = D == 128 ? 128 : 64;
  static constexpr int QT = kAttnQTile;
  static constexpr int CTAS = D == 128 ? 1 : 2;
  static constexpr int NST = D == 128 ? 2 : D == 64 ? 4 : 6;
  static constexpr int Q_B = Tile::bytes(QT), KV_B = Tile::bytes(KT);
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * Q_B;
  static constexpr int OFF_V = OFF_K + NST * KV_B;
  static constexpr int OFF_BAR = OFF_V + NST * KV_B;
  static constexpr int N_BAR = 2 + 2 * NST + 2 + 2 + 2 + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * N_BAR;
  static constexpr int BYTES = OFF_MISC + 32 + 4 * NST;
  static constexpr uint32_t COL_S = 0, COL_O = 2 * KT;
  static constexpr uint32_t TMEM_COLS = COL_O + 2 * D <= 256 ? 256 : 512;
  static constexpr int THREADS = 320;   // warps 0-3, 4-7: softmax; 8: loads; 9: MMAs
  static_assert(COL_O + 2 * D <= TMEM_COLS && TMEM_COLS * CTAS <= 512, "TMEM columns");
  static_assert(KV_B % 1024 == 0 && Q_B % 1024 == 0, "tiles hold whole swizzle atoms");
};

// Key tiles [a, b) that rows [r0, r0 + 128) see.
__device__ __forceinline__ int2 tile_range(const BatchMask& m, int r0, int KT) {
  const int r1 = min(r0 + kAttnQTile, m.qlen);
  if (r0 >= r1) return make_int2(0, 0);
  const int lo = row_interval(m, r0).x, hi = row_interval(m, r1 - 1).y;
  return lo < hi ? make_int2(lo / KT, (hi + KT - 1) / KT) : make_int2(0, 0);
}

template <int D, bool MOD>
__global__ void __launch_bounds__(FwdCfg<D>::THREADS, FwdCfg<D>::CTAS)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const AttnParams p) {
  using Cfg = FwdCfg<D>;
  using Tile = RowTile<D>;
  constexpr int KT = Cfg::KT, QT = Cfg::QT, NST = Cfg::NST;
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
  volatile int* range = reinterpret_cast<volatile int*>(sm + Cfg::OFF_MISC + 8);       // [4]
  volatile int* last_load = reinterpret_cast<volatile int*>(sm + Cfg::OFF_MISC + 32);  // [NST]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int BH = p.B * p.Hq, n_qt = gridDim.x / BH;
  // the last query tiles see the most keys under a causal mask: first
  const int qt = n_qt - 1 - static_cast<int>(blockIdx.x) / BH, bh = static_cast<int>(blockIdx.x) % BH;
  const int b = bh / p.Hq, h = bh % p.Hq, hk = h / p.G;
  const int q0 = qt * 2 * QT, split = blockIdx.y;
  const BatchMask mask = batch_mask(p.mask, b);

  if (threadIdx.x < 2) {
    const int2 r = tile_range(mask, q0 + threadIdx.x * QT, KT);
    range[2 * threadIdx.x] = r.x;
    range[2 * threadIdx.x + 1] = r.y;
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
  if (warp == 9) {
    tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{p.err, abort_flag, p.timeout_ns};

  // this split's key tiles [jlo, jhi), and of them each query tile's [a, b)
  int a[2] = {range[0], range[2]}, e[2] = {range[1], range[3]};
  int jlo, jhi;
  {
    const bool live0 = a[0] < e[0], live1 = a[1] < e[1];
    jlo = live0 && live1 ? min(a[0], a[1]) : live0 ? a[0] : a[1];
    jhi = live0 && live1 ? max(e[0], e[1]) : live0 ? e[0] : e[1];
    const int per = (jhi - jlo + p.splits - 1) / p.splits;
    jlo = min(jhi, jlo + split * per);
    jhi = min(jhi, jlo + per);
    for (int w = 0; w < 2; ++w) {
      a[w] = max(a[w], jlo);
      e[w] = min(e[w], jhi);
      if (a[w] >= e[w]) a[w] = e[w] = 0;
    }
  }
  const int ntiles = jhi - jlo;

  if (warp == 8) {
    // ------------------------------------------------------------ loads
    if (lane == 0 && ntiles > 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      for (int w = 0; w < 2; ++w) {
        mbar_arrive_expect_tx(q_full + w, Cfg::Q_B);   // rows behind the tensor's last come as zeros
        Tile::load(sq + w * Cfg::Q_B, &tm_q, q_full + w, q0 + w * QT, h, b, QT);
      }
      for (int n = 0; n < ntiles; ++n) {
        const int st = n % NST;
        if (n >= NST && !mbar_wait(kv_empty + st, (n / NST - 1) & 1, wc)) break;
        mbar_arrive_expect_tx(kv_full + st, 2 * Cfg::KV_B);
        Tile::load(sk + st * Cfg::KV_B, &tm_k, kv_full + st, (jlo + n) * KT, hk, b, KT);
        Tile::load(sv + st * Cfg::KV_B, &tm_v, kv_full + st, (jlo + n) * KT, hk, b, KT);
        last_load[st] = n;
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMAs
    if (lane == 0 && ntiles > 0) {
      const uint32_t idesc_s = idesc_bf16_f32(128, KT, false, false);
      const uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
      const uint64_t k_desc = Tile::desc_k(sk), v_desc = Tile::desc_mn(sv, KT);
      auto issue_s = [&](int w, int n) -> bool {   // scores of tile n
        const int st = n % NST;
        if (!mbar_wait_mma(kv_full + st, (n / NST) & 1, wc)) return false;
        tc_fence_after();
        const uint64_t qd = Tile::desc_k(sq + w * Cfg::Q_B);
        const uint64_t kd = k_desc + static_cast<uint64_t>((st * Cfg::KV_B) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss(tmem + Cfg::COL_S + w * KT, qd + Tile::kstep_k(kk, QT), kd + Tile::kstep_k(kk, KT), idesc_s,
                  kk > 0 ? 1u : 0u);
        umma_commit(s_full + w);
        return true;
      };
      bool ok = mbar_wait_mma(q_full, 0, wc) && mbar_wait_mma(q_full + 1, 0, wc);
      int used[2] = {0, 0};
      for (int w = 0; ok && w < 2; ++w)
        if (a[w] < e[w] && a[w] == jlo) ok = issue_s(w, 0);
      for (int n = 0; ok && n < ntiles; ++n) {
        const int j = jlo + n, st = n % NST;
        for (int w = 0; ok && w < 2; ++w) {
          if (j >= a[w] && j < e[w]) {
            if (!mbar_wait_mma(p_full + w, used[w]++ & 1, wc)) { ok = false; break; }
            tc_fence_after();
            const uint64_t vd = v_desc + static_cast<uint64_t>((st * Cfg::KV_B) >> 4);
#pragma unroll
            for (int ks = 0; ks < KT / 16; ++ks)
              umma_ts(tmem + Cfg::COL_O + w * D, tmem + Cfg::COL_S + w * KT + ks * 8, vd + ks * Tile::KSTEP_MN, idesc_o,
                      (j > a[w] || ks > 0) ? 1u : 0u);
            if (j + 1 == e[w]) umma_commit(o_full + w);
          }
          if (j + 1 >= a[w] && j + 1 < e[w]) ok = issue_s(w, n + 1);
        }
        umma_commit(kv_empty + st);
      }
      umma_commit(all_done);   // every MMA issued above is done
      mbar_wait_drain(all_done, 0, p.timeout_ns);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int w = warp >> 2, wq = warp & 3;
    const int tid = threadIdx.x & 127;              // row of the tile; also the key whose V row it may zero
    const int row = q0 + w * QT + tid;
    const int2 iv = row < p.mask.Nq ? row_interval(mask, row) : make_int2(0, 0);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t col_s = lane_base + Cfg::COL_S + w * KT, col_o = lane_base + Cfg::COL_O + w * D;
    const float c2 = p.scale * kLog2e;
    const float tanh_in = MOD && p.cap > 0.f ? 2.f * c2 / p.cap : 0.f, tanh_out = p.cap * kLog2e;
    const float slope2 = MOD && p.slopes ? p.slopes[h] * kLog2e : 0.f;
    const int pos = bias_position(mask, row, iv);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const int n_w = e[w] - a[w];
    for (int it = 0; it < n_w; ++it) {
      const int j = a[w] + it, k0 = j * KT, n = j - jlo, st = n % NST;
      // the V row this thread answers for: a key that no query may see
      bool dead = false;
      if (KT == 128 || tid < KT) {
        const int key = k0 + tid;
        dead = key >= mask.len && key < mask.nk;
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
      if (MOD) {
        if (p.cap > 0.f) {
#pragma unroll
          for (int k = 0; k < KT; ++k) s[k] = __float_as_uint(tanh_exp(__uint_as_float(s[k]) * tanh_in) * tanh_out);
        } else {
#pragma unroll
          for (int k = 0; k < KT; ++k) s[k] = __float_as_uint(__uint_as_float(s[k]) * c2);
        }
        if (p.slopes) {
          const int d0 = pos - k0;
#pragma unroll
          for (int k = 0; k < KT; ++k)
            s[k] = __float_as_uint(fmaf(-slope2, fabsf(static_cast<float>(d0 - k)), __uint_as_float(s[k])));
        }
      }
      if (!__all_sync(~0u, iv.x <= k0 && iv.y >= k0 + KT)) {
        const int first = iv.x - k0, last = iv.y - k0;
#pragma unroll
        for (int k = 0; k < KT; ++k)
          if (k < first || k >= last) s[k] = 0xFF800000u;   // -inf
      }
      float mx = __uint_as_float(s[0]);
#pragma unroll
      for (int k = 1; k < KT; ++k) mx = fmaxf(mx, __uint_as_float(s[k]));
      if (!MOD) mx *= c2;
      if (it == 0) {
        m = mx;
      } else if (__any_sync(~0u, mx > m + 8.f)) {
        const float m_new = fmaxf(m, mx);
        const float f = m == -INFINITY ? 0.f : ex2_mufu(m - m_new);
        m = m_new;
        l *= f;
#pragma unroll
        for (int d = 0; d < D; d += 16) {
          uint32_t o[16];
          tmem_ld16(col_o + d, o);
          tmem_wait_ld();
          regs_loaded(o);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st16(col_o + d, o);
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < KT; c += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float s0 = __uint_as_float(s[c + 2 * k]), s1 = __uint_as_float(s[c + 2 * k + 1]);
          const float p0 = ex2_mufu(MOD ? s0 - base : fmaf(s0, c2, -base));
          const float p1 = ex2_mufu(MOD ? s1 - base : fmaf(s1, c2, -base));
          sum += p0 + p1;
          pk[k] = pack_bf16x2(p0, p1);
        }
        tmem_st16(col_s + c / 2, pk);
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
    ok = __all_sync(~0u, ok);
    if (ok && q0 + w * QT + wq * 32 < p.mask.Nq) {
      tc_fence_after();
      const bool have = row < p.mask.Nq;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const float lse2 = l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;   // l: NaN
      const long at = (static_cast<long>(b) * p.Hq + h) * p.mask.Nq + row;
      const long part_row = static_cast<long>(split) * BH * p.mask.Nq + at;
      if (have) {
        if (p.splits > 1) p.part_l[part_row] = lse2;
        else if (p.L)
          p.L[at] = lse2 * 0.69314718055994531f - (MOD && p.slopes && l > 0.f ? p.slopes[h] * bias_shift(mask, row, iv) : 0.f);
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
        if (have) {
          if (p.splits > 1) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + part_row * D + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(y + d);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              dst[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                  pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8 && lane == 0 && ntiles > 0) {   // copies still in flight (only after an abort) must land before exit
    for (int st = 0; st < NST; ++st)
      if (last_load[st] >= 0) mbar_wait_drain(kv_full + st, (last_load[st] / NST) & 1, p.timeout_ns);
    for (int w = 0; w < 2; ++w) mbar_wait_drain(q_full + w, 0, p.timeout_ns);
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::TMEM_COLS);
  }
}

// Join of the splits of one row (one warp a row): weights 2^(l_s - max).
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnParams p) {
  const long rows = static_cast<long>(p.B) * p.Hq * p.mask.Nq;
  const long at = static_cast<long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (at >= rows) return;
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, p.part_l[s * rows + at]);
  const float base = top == -INFINITY ? 0.f : top;
  float total = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < p.splits; ++s) {
    const float w = ex2_mufu(p.part_l[s * rows + at] - base);
    total += w;
    const float* o = p.part_o + (s * rows + at) * p.D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < p.D) acc[i] = fmaf(w, o[lane + 32 * i], acc[i]);
  }
  const int n = static_cast<int>(at % p.mask.Nq);
  const long bh = at / p.mask.Nq;
  const int b = static_cast<int>(bh / p.Hq), h = static_cast<int>(bh % p.Hq);
  uint16_t* y = p.y + b * p.ys[0] + h * p.ys[1] + n * p.ys[2];
  const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < p.D) y[lane + 32 * i] = static_cast<uint16_t>(pack_bf16x2(acc[i] * inv, 0.f));
  if (lane == 0 && p.L) {
    float L = total == 0.f ? -INFINITY : (top + log2f(total)) * 0.69314718055994531f;
    if (p.slopes && total > 0.f) {
      const BatchMask m = batch_mask(p.mask, b);
      L -= p.slopes[h] * bias_shift(m, n, row_interval(m, n));
    }
    p.L[at] = L;
  }
}

// Documents: the start and the end of the run of equal ids each position lies
// in.  One CTA a batch entry; two passes of a running maximum (of the last
// position where a run began) and a running minimum from the right.
constexpr int kDocThreads = 1024, kDocPer = 8;
template <bool MAX>
__device__ __forceinline__ int block_scan(int v, int* sh) {   // inclusive, over the block, in thread order
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = MAX ? __shfl_up_sync(~0u, v, o) : __shfl_down_sync(~0u, v, o);
    if (MAX ? lane >= o : lane + o < 32) v = MAX ? max(v, u) : min(v, u);
  }
  if (lane == (MAX ? 31 : 0)) sh[warp] = v;
  __syncthreads();
  int t = sh[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = MAX ? __shfl_up_sync(~0u, t, o) : __shfl_down_sync(~0u, t, o);
    if (MAX ? lane >= o : lane + o < 32) t = MAX ? max(t, u) : min(t, u);
  }
  const int other = __shfl_sync(~0u, t, MAX ? max(warp - 1, 0) : min(warp + 1, 31));
  if (MAX ? warp > 0 : warp < 31) v = MAX ? max(v, other) : min(v, other);
  __syncthreads();
  return v;
}
__global__ void __launch_bounds__(kDocThreads) attn_documents_kernel(const int32_t* ids, int2* doc, int N) {
  __shared__ int sh[32];
  __shared__ int carry;
  ids += static_cast<long>(blockIdx.x) * N;
  doc += static_cast<long>(blockIdx.x) * N;
  constexpr int STEP = kDocThreads * kDocPer;
  const int chunks = (N + STEP - 1) / STEP;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  for (int c = 0; c < chunks; ++c) {
    const int i0 = c * STEP + threadIdx.x * kDocPer;   // N < 2^30
    int start[kDocPer], run = -1;
#pragma unroll
    for (int k = 0; k < kDocPer; ++k) {
      const int i = i0 + k;
      if (i < N && (i == 0 || ids[i] != ids[i - 1])) run = i;
      start[k] = run;
    }
    const int before = block_scan<true>(run, sh);
    int prev = __shfl_up_sync(~0u, before, 1);
    if ((threadIdx.x & 31) == 31) sh[threadIdx.x >> 5] = before;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) prev = threadIdx.x == 0 ? -1 : sh[(threadIdx.x >> 5) - 1];
    prev = max(prev, carry);
#pragma unroll
    for (int k = 0; k < kDocPer; ++k)
      if (i0 + k < N) doc[i0 + k].x = max(start[k], prev);
    __syncthreads();
    if (threadIdx.x == kDocThreads - 1) carry = max(carry, before);
    __syncthreads();
  }
  if (threadIdx.x == 0) carry = N;
  __syncthreads();
  for (int c = chunks - 1; c >= 0; --c) {
    const int i0 = c * STEP + threadIdx.x * kDocPer;
    int end[kDocPer], run = N;
#pragma unroll
    for (int k = kDocPer - 1; k >= 0; --k) {
      const int i = i0 + k;
      if (i + 1 < N && ids[i + 1] != ids[i]) run = i + 1;
      end[k] = run;
    }
    const int after = block_scan<false>(run, sh);
    int next = __shfl_down_sync(~0u, after, 1);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = after;
    __syncthreads();
    if ((threadIdx.x & 31) == 31) next = threadIdx.x == kDocThreads - 1 ? N : sh[(threadIdx.x >> 5) + 1];
    next = min(next, carry);
#pragma unroll
    for (int k = 0; k < kDocPer; ++k) {
      const int i = i0 + k;
      if (i < N) doc[i].y = ids[i] < 0 ? doc[i].x : min(end[k], next);
    }
    __syncthreads();
    if (threadIdx.x == 0) carry = min(carry, after);
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_attn_documents(const int32_t* ids, int2* doc, int B, int N, cudaStream_t s) {
  attn_documents_kernel<<<B, kDocThreads, 0, s>>>(ids, doc, N);
  return cudaGetLastError();
}

int attn_fwd_key_tile(int D) { return D == 128 ? FwdCfg<128>::KT : FwdCfg<64>::KT; }

cudaError_t launch_attn_fwd(const AttnMaps& m, const AttnParams& p, cudaStream_t s) {
  const int n_qt = (p.mask.Nq + 2 * kAttnQTile - 1) / (2 * kAttnQTile);
  const dim3 grid(static_cast<unsigned>(static_cast<long>(n_qt) * p.B * p.Hq), static_cast<unsigned>(p.splits));
  auto go = [&](auto kern, int bytes, int threads, int ctas) {
    // at most `ctas` CTAs share an SM, so that each finds its TMEM columns free
    const int floor = 228 * 1024 / (ctas + 1) + 1024;
    const int smem = bytes + 1024 > floor ? bytes + 1024 : floor;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<grid, threads, smem, s>>>(m.q, m.k, m.v, p);
    return cudaGetLastError();
  };
  const bool mod = p.cap > 0.f || p.slopes;
  auto by_mod = [&](auto d) {
    constexpr int D = decltype(d)::value;
    using C = FwdCfg<D>;
    return mod ? go(attn_fwd_kernel<D, true>, C::BYTES, C::THREADS, C::CTAS)
               : go(attn_fwd_kernel<D, false>, C::BYTES, C::THREADS, C::CTAS);
  };
  switch (p.D) {
    case 16: return by_mod(std::integral_constant<int, 16>{});
    case 32: return by_mod(std::integral_constant<int, 32>{});
    case 64: return by_mod(std::integral_constant<int, 64>{});
    case 128: return by_mod(std::integral_constant<int, 128>{});
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_attn_join(const AttnParams& p, cudaStream_t s) {
  const long rows = static_cast<long>(p.B) * p.Hq * p.mask.Nq;
  attn_join_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace flare
