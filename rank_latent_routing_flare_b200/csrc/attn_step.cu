// Exact softmax attention of few query rows: single new tokens over a long
// cache.  A key head's query rows (its G query heads times Nq <= 16 rows)
// share every key and value, so K and V are read once and the kernel is bound
// by HBM; the products (m16n8k16 mma.sync, 16 rows at a time) are far below
// the tensor pipe's rate and take registers as they come from global memory.
//
// Each warp streams chunks of 16 keys, 16-byte loads straight into the
// operand fragments, the next chunk's loads in flight while one is computed:
//  - scores: a lane's 8 consecutive elements of a K row feed two k-steps; the
//    order of D inside a dot product is free, and Q's fragments use the same.
//  - values: lane (g, t) reads elements 8g .. 8g+7 of the four V rows 2t, 2t+1,
//    2t+8, 2t+9 and pairs rows with byte permutes; output column n of product i
//    is element 8n + i.
// Rows keep a running reference and sum as in the tiled kernel.  The keys are
// split over CTAs, within a CTA over 8 warps, which join in shared memory; up
// to eight splits are a cluster and join there too.
#include <type_traits>
#include <utility>

#include "attn_common.cuh"
#include "ops_internal.h"

namespace flare {
namespace {

constexpr int kStepWarps = 8, kChunk = 16;

struct StepParams {
  AttnParams a;
  AttnSide q, k, v;
};

template <int D>
struct StepCfg {
  static constexpr int KB = D >= 32 ? D / 32 : 1;   // loads per K row and lane
  static constexpr int KE = D >= 32 ? 8 : 4;        // elements per load
  static constexpr int VE = D >= 64 ? 8 : D / 8;
  static constexpr int VB = D / (8 * VE);
};

template <int N>   // words of 4 bytes
__device__ __forceinline__ void load_words(const uint16_t* p, bool ok, uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = 0u;
  if (!ok) return;
  if constexpr (N == 4)
    asm("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
  else if constexpr (N == 2)
    asm("ld.global.nc.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  else
    asm("ld.global.nc.L1::no_allocate.b32 %0, [%1];" : "=r"(w[0]) : "l"(p));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
struct Chunk {
  uint32_t k[2][StepCfg<D>::KB][StepCfg<D>::KE / 2];   // keys g and 8 + g
  uint32_t v[4][StepCfg<D>::VB][StepCfg<D>::VE / 2];   // keys 2t, 2t+1, 2t+8, 2t+9
};
template <int D>
__device__ __forceinline__ void load_chunk(Chunk<D>& c, const StepParams& p, const BatchMask& m, const uint16_t* kb,
                                           const uint16_t* vb, int key0, int end) {
  using C = StepCfg<D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int key = key0 + 8 * n + g;
#pragma unroll
    for (int i = 0; i < C::KB; ++i)
      load_words(kb + static_cast<long>(key) * p.k.sn + 32 * i + C::KE * t, key < end, c.k[n][i]);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int key = key0 + 2 * t + (r & 1) + 8 * (r >> 1);
    bool ok = key < end;
    if (m.doc && ok) {   // a weight of 0 does not erase a NaN: padding inside the range is not read
      const int2 d = m.doc[key];
      ok = d.x != d.y;
    }
#pragma unroll
    for (int i = 0; i < C::VB; ++i)
      load_words(vb + static_cast<long>(key) * p.v.sn + 64 * i + C::VE * g, ok, c.v[r][i]);
  }
}

// CAP: capped scores; without, the tanh's coefficients take no registers.
template <int D, bool CAP>
__global__ void __launch_bounds__(kStepWarps * 32, D == 128 ? 1 : 2) attn_step_kernel(const StepParams p) {
  using C = StepCfg<D>;
  extern __shared__ __align__(16) float sh[];   // [warps][rows] (m, l) pairs, then [warps][rows][D]
  const AttnParams& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x % a.splits, bk = blockIdx.x / a.splits, b = bk / a.Hk, hk = bk % a.Hk;
  const int rows = a.G * a.mask.Nq;
  const BatchMask mask = batch_mask(a.mask, b);

  // the keys that any row sees, rounded to chunks and dealt to the splits
  int lo = 0, hi = 0;
  const int last_row = min(a.mask.Nq, mask.qlen) - 1;
  if (blockIdx.x == 0 && threadIdx.x < 4) a.err[threadIdx.x] = 0u;   // nothing here can wait in vain
  if (last_row >= 0) {
    lo = row_interval(mask, 0).x / kChunk * kChunk;
    hi = row_interval(mask, last_row).y;
  }
  const int chunks = hi > lo ? (hi - lo + kChunk - 1) / kChunk : 0;
  const int per = (chunks + a.splits - 1) / a.splits;
  const int c_end = min(chunks, (split + 1) * per);

  // this lane's two rows: r = i G + head
  int2 iv[2];
  int pos[2];
  float slope2[2];
  __shared__ uint4 sm_q[D / 16][32];   // Q's operand fragments, the same for every warp: read per chunk, they hold no registers
  uint32_t qf[D / 16][4];
  const ScoreOps ops(a.scale, a.cap, true);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = g + 8 * u, i = r / a.G, h = hk * a.G + r % a.G;
    const bool have = r < rows;
    iv[u] = have ? row_interval(mask, i) : make_int2(0, 0);
    pos[u] = bias_position(mask, have ? i : 0, iv[u]);
    slope2[u] = have && a.slopes ? a.slopes[h] * kLog2e : 0.f;
    const uint16_t* q = p.q.p + b * p.q.sb + h * p.q.sh + static_cast<long>(i) * p.q.sn;
#pragma unroll
    for (int blk = 0; blk < C::KB; ++blk) {
      uint32_t w[C::KE / 2];
      load_words(q + 32 * blk + C::KE * t, have, w);
#pragma unroll
      for (int s = 0; s < C::KE / 4; ++s) {
        qf[blk * (C::KE / 4) + s][u] = w[2 * s];
        qf[blk * (C::KE / 4) + s][2 + u] = w[2 * s + 1];
      }
    }
  }
  if (warp == 0) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) sm_q[k][lane] = make_uint4(qf[k][0], qf[k][1], qf[k][2], qf[k][3]);
  }
  __syncthreads();
  const uint16_t* kb = p.k.p + b * p.k.sb + hk * p.k.sh;
  const uint16_t* vb = p.v.p + b * p.v.sb + hk * p.v.sh;

  float o[C::VB][C::VE][4];
#pragma unroll
  for (int i = 0; i < C::VB; ++i)
#pragma unroll
    for (int j = 0; j < C::VE; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][j][k] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  auto compute = [&](const Chunk<D>& c, int key0) {
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[n][k] = 0.f;
#pragma unroll
    for (int blk = 0; blk < C::KB; ++blk)
#pragma unroll
      for (int u = 0; u < C::KE / 4; ++u) {
        uint32_t q[4];
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3])
                     : "r"(smem_u32(&sm_q[blk * (C::KE / 4) + u][lane])));
#pragma unroll
        for (int n = 0; n < 2; ++n) mma16816(s[n], q, c.k[n][blk][2 * u], c.k[n][blk][2 * u + 1]);
      }
    float mx[2] = {-INFINITY, -INFINITY};
    if (CAP) {
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(s[0][k]), fabsf(s[1][k])));
      if (__all_sync(~0u, ops.small(top))) {
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          float* x = &s[k / 4][k % 4];
          f2_unpack(ops.poly(f2_pack(x[0], x[1]), f2_dup(0.f)), x[0], x[1]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k / 4][k % 4] = ops.capped(s[k / 4][k % 4]);
      }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int u = k >> 1, key = key0 + 8 * n + 2 * t + (k & 1);
        float x = CAP ? s[n][k] : s[n][k] * ops.c2;
        if (a.slopes) x = fmaf(-slope2[u], fabsf(static_cast<float>(pos[u] - key)), x);
        if (key < iv[u].x || key >= iv[u].y) x = -INFINITY;
        s[n][k] = x;
        mx[u] = fmaxf(mx[u], x);
      }
    if (__any_sync(~0u, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
      float f[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        mx[u] = fmaxf(mx[u], __shfl_xor_sync(~0u, mx[u], 1));
        mx[u] = fmaxf(mx[u], __shfl_xor_sync(~0u, mx[u], 2));
        const float m_new = fmaxf(m[u], mx[u]);
        f[u] = m[u] == -INFINITY ? 0.f : ex2_mufu(m[u] - m_new);
        m[u] = m_new;
        l[u] *= f[u];
      }
#pragma unroll
      for (int i = 0; i < C::VB; ++i)
#pragma unroll
        for (int j = 0; j < C::VE; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][j][k] *= f[k >> 1];
    }
    uint32_t pf[4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float base = m[u] == -INFINITY ? 0.f : m[u];
        const float p0 = ex2_mufu(s[n][2 * u] - base), p1 = ex2_mufu(s[n][2 * u + 1] - base);
        l[u] += p0 + p1;
        pf[2 * n + u] = pack_bf16x2(p0, p1);
      }
#pragma unroll
    for (int i = 0; i < C::VB; ++i)
#pragma unroll
      for (int j = 0; j < C::VE; ++j) {
        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
        mma16816(o[i][j], pf, __byte_perm(c.v[0][i][j / 2], c.v[1][i][j / 2], sel),
                 __byte_perm(c.v[2][i][j / 2], c.v[3][i][j / 2], sel));
      }
  };

  Chunk<D> buf[2];
  int c = split * per + warp;
  if (c < c_end) load_chunk<D>(buf[0], p, mask, kb, vb, lo + c * kChunk, hi);
  for (; c < c_end; c += 2 * kStepWarps) {
    const int next = c + kStepWarps;
    if (next < c_end) load_chunk<D>(buf[1], p, mask, kb, vb, lo + next * kChunk, hi);
    compute(buf[0], lo + c * kChunk);
    if (next >= c_end) break;
    if (next + kStepWarps < c_end) load_chunk<D>(buf[0], p, mask, kb, vb, lo + (next + kStepWarps) * kChunk, hi);
    compute(buf[1], lo + next * kChunk);
  }

  // join the warps: row statistics, then the outputs
  float* sm_ml = sh;
  float* sm_o = sh + 2 * kStepWarps * rows;
  // a cluster's partial outputs and log2 sums, behind the warps'
  float* sm_part = sm_o + kStepWarps * rows * D;
  float* sm_lse = sm_part + rows * (D + 4);
  const bool in_cluster = a.splits > 1 && a.splits <= kAttnClusterSplits;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    l[u] += __shfl_xor_sync(~0u, l[u], 1);
    l[u] += __shfl_xor_sync(~0u, l[u], 2);
    const int r = g + 8 * u;
    if (r < rows) {
      if (t == 0) {
        sm_ml[2 * (warp * rows + r)] = m[u];
        sm_ml[2 * (warp * rows + r) + 1] = l[u];
      }
#pragma unroll
      for (int i = 0; i < C::VB; ++i)
#pragma unroll
        for (int j = 0; j < C::VE; ++j) {
          float* d = sm_o + (warp * rows + r) * D + 64 * i + j;
          d[2 * t * C::VE] = o[i][j][2 * u];
          d[(2 * t + 1) * C::VE] = o[i][j][2 * u + 1];
        }
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < rows * (D / 2); idx += blockDim.x) {
    const int r = idx / (D / 2), d = 2 * (idx % (D / 2));
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kStepWarps; ++w) top = fmaxf(top, sm_ml[2 * (w * rows + r)]);
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll
    for (int w = 0; w < kStepWarps; ++w) {
      const float f = ex2_mufu(sm_ml[2 * (w * rows + r)] - base);
      const float2 v = *reinterpret_cast<const float2*>(sm_o + (w * rows + r) * D + d);
      total = fmaf(sm_ml[2 * (w * rows + r) + 1], f, total);
      x0 = fmaf(v.x, f, x0);
      x1 = fmaf(v.y, f, x1);
    }
    const int i = r / a.G, h = hk * a.G + r % a.G;
    const long at = (static_cast<long>(b) * a.Hq + h) * a.mask.Nq + i;
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const float lse2 = total == 0.f ? -INFINITY : top + log2f(total);
    if (in_cluster) {
      *reinterpret_cast<float2*>(sm_part + r * (D + 4) + d) = make_float2(x0 * inv, x1 * inv);
      if (d == 0) sm_lse[r] = lse2;
    } else if (a.splits > 1) {
      const long part = static_cast<long>(split) * a.B * a.Hq * a.mask.Nq + at;
      *reinterpret_cast<float2*>(a.part_o + part * D + d) = make_float2(x0 * inv, x1 * inv);
      if (d == 0) a.part_l[part] = lse2;
    } else {
      *reinterpret_cast<uint32_t*>(a.y + b * a.ys[0] + h * a.ys[1] + i * a.ys[2] + d) = pack_bf16x2(x0 * inv, x1 * inv);
      if (d == 0 && a.L) a.L[at] = natural_lse(a, mask, h, i, lse2);
    }
  }
  if (in_cluster) {
    cluster_sync();
    cluster_join<D, D + 4>(a.splits, split, sm_part, sm_lse, rows, threadIdx.x, blockDim.x, [&](int r, int d, float4 v, float lse2) {
      const int i = r / a.G, h = hk * a.G + r % a.G;
      *reinterpret_cast<uint2*>(a.y + b * a.ys[0] + h * a.ys[1] + i * a.ys[2] + d) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      if (d == 0 && a.L) a.L[(static_cast<long>(b) * a.Hq + h) * a.mask.Nq + i] = natural_lse(a, mask, h, i, lse2);
    });
    __syncwarp();
    cluster_sync();   // the others have read this CTA's rows
  }
}

// Row statistics and outputs of the warps, and of the CTA for its cluster.
constexpr int step_smem(int rows, int D) { return 4 * rows * (kStepWarps * (D + 2) + D + 5); }

}  // namespace

cudaError_t launch_attn_step(const AttnParams& p, const AttnSide& q, const AttnSide& k, const AttnSide& v,
                             cudaStream_t s) {
  const StepParams sp{p, q, k, v};
  const dim3 grid(static_cast<unsigned>(static_cast<long>(p.splits) * p.B * p.Hk));
  const int rows = p.G * p.mask.Nq, smem = step_smem(rows, p.D);
  auto go = [&](auto d, auto cap) {
    constexpr int D = decltype(d)::value;
    auto* kern = attn_step_kernel<D, decltype(cap)::value>;
    if (smem > 48 * 1024) {
      const cudaError_t e = allow_smem<std::pair<StepCfg<D>, decltype(cap)>>(kern, step_smem(kAttnStepRows, D));
      if (e != cudaSuccess) return e;
    }
    return launch_splits(kern, grid, kStepWarps * 32, smem, s, dim3(p.splits, 1, 1), p.splits, sp);
  };
  auto by_cap = [&](auto d) { return p.cap > 0.f ? go(d, std::true_type{}) : go(d, std::false_type{}); };
  switch (p.D) {
    case 16: return by_cap(std::integral_constant<int, 16>{});
    case 32: return by_cap(std::integral_constant<int, 32>{});
    case 64: return by_cap(std::integral_constant<int, 64>{});
    case 128: return by_cap(std::integral_constant<int, 128>{});
  }
  return cudaErrorInvalidValue;
}

}  // namespace flare
