// Device code shared by the attention kernels: masks, score modifiers and the
// layout of row tiles in shared memory.
#pragma once

#include "attention.h"
#include "attn_math.cuh"
#include "ptx.cuh"

namespace flare {

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// Untiled copy of `bytes` (a multiple of 16, both addresses 16-byte aligned).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

constexpr float kLog2e = 1.4426950408889634f;

// Masks of one batch entry.
struct BatchMask {
  int len, qlen, pre, causal, nk;
  long off;
  const int2* doc;
};
__device__ __forceinline__ BatchMask batch_mask(const AttnMask& m, int b) {
  BatchMask r;
  r.nk = m.Nk;
  r.len = m.lengths ? max(0, min(m.Nk, m.lengths[b])) : m.Nk;
  r.qlen = m.q_lengths ? max(0, min(m.Nq, m.q_lengths[b])) : m.Nq;
  r.off = m.q_offsets ? static_cast<long>(m.q_offsets[b]) : static_cast<long>(m.Nk) - m.Nq;
  r.pre = m.prefix ? m.prefix[b] : 0;
  r.causal = m.causal;
  r.doc = m.doc ? m.doc + static_cast<long>(b) * m.Nk : nullptr;
  return r;
}
// Keys [x, y) that row i sees (x = y: none).  Neither end lies behind the
// length, not for a row that sees nothing either: kernels visit what lies
// between the first row's and the last row's ends, and that is no padding.
__device__ __forceinline__ int2 row_interval(const BatchMask& m, int i) {
  const long p = m.off + i;
  long lo = 0, hi = m.len;
  if (m.causal) hi = min(hi, max(max(p + 1, static_cast<long>(m.pre)), 0L));
  if (m.doc) {
    if (p < 0) {
      hi = 0;
    } else if (p >= m.nk) {
      lo = hi = m.len;
    } else {
      const int2 d = m.doc[p];
      lo = min(d.x, m.len);
      hi = min(hi, static_cast<long>(d.y));
    }
  }
  if (hi < lo || i >= m.qlen) hi = lo;
  return make_int2(static_cast<int>(lo), static_cast<int>(hi));
}
// Position of row i for the distance bias, moved to the nearest key it sees:
// |p - j| = |p - p'| + |p' - j| for every such key j, and the softmax does
// not see the first term.  Distances stay exact in fp32 that way, however
// far the row stands from its keys.
__device__ __forceinline__ int bias_position(const BatchMask& m, int i, int2 iv) {
  const long p = m.off + i;
  return static_cast<int>(max(static_cast<long>(iv.x), min(p, static_cast<long>(iv.y) - 1)));
}
__device__ __forceinline__ float bias_shift(const BatchMask& m, int i, int2 iv) {   // |p - p'|
  const long d = m.off + i - bias_position(m, i, iv);
  return static_cast<float>(d < 0 ? -d : d);
}

// One lane of a converged warp, the same at every call.  The MMA warps run
// their loops converged, with warp-uniform descriptors, and only issue under
// this: an MMA issued from a branch on the lane number took about 80 clocks,
// its operands having to be made uniform one by one.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(ok));
  return ok != 0;
}

// Registers of the executing warpgroup (all of its warps).
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Clusters: every thread of every CTA arrives, whatever became of its own waits.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_smem(const void* p, int rank) {   // the same address in another CTA of the cluster
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float peer_load(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_load4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
// Join of a cluster's splits (CTA rank = split): every CTA holds `rows` rows of
// normalised outputs (STRIDE floats apart) and their log2 sums; each CTA joins
// its share of the rows and hands them to out(row, first column, four values,
// log2 sum).  `threads` threads call it, numbered by `t`, between two
// cluster_sync of all.
template <int D, int STRIDE, typename Out>
__device__ __forceinline__ void cluster_join(int splits, int rank, const float* part, const float* lse, int rows, int t,
                                             int threads, Out&& out) {
  const int per = (rows + splits - 1) / splits, r0 = rank * per, r1 = min(rows, r0 + per);
  for (int i = t; i < (r1 - r0) * (D / 4); i += threads) {
    const int row = r0 + i / (D / 4), d = 4 * (i % (D / 4));
    float l[kAttnClusterSplits], top = -INFINITY;
#pragma unroll
    for (int s = 0; s < kAttnClusterSplits; ++s) {
      l[s] = s < splits ? peer_load(peer_smem(lse + row, s)) : -INFINITY;
      top = fmaxf(top, l[s]);
    }
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < kAttnClusterSplits; ++s)
      if (s < splits) {
        const float w = ex2_mufu(l[s] - base);
        const float4 v = peer_load4(peer_smem(part + row * STRIDE + d, s));
        total += w;
        a.x = fmaf(w, v.x, a.x);
        a.y = fmaf(w, v.y, a.y);
        a.z = fmaf(w, v.z, a.z);
        a.w = fmaf(w, v.w, a.w);
      }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    out(row, d, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv), total == 0.f ? -INFINITY : top + log2f(total));
  }
}
// log-sum-exp of a row in natural units, from its log2 sum over biased positions.
__device__ __forceinline__ float natural_lse(const AttnParams& p, const BatchMask& m, int h, int row, float lse2) {
  float L = lse2 * 0.69314718055994531f;
  if (p.slopes && lse2 != -INFINITY) L -= p.slopes[h] * bias_shift(m, row, row_interval(m, row));
  return L;
}

// After tcgen05.wait::ld: the registers a TMEM load wrote are defined here,
// so that no use of them is scheduled before the wait.
template <int N>
__device__ __forceinline__ void regs_loaded(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Row tiles in shared memory: panels of up to 64 elements (128 bytes, the
// widest swizzle), each `rows` x PANEL elements as TMA writes them.
template <int D>
struct RowTile {
  static constexpr int PANEL = D < 64 ? D : 64;
  static constexpr int NP = D / PANEL;
  static constexpr int ROWB = PANEL * 2;
  static constexpr uint32_t LAYOUT = ROWB == 32 ? LAYOUT_SW32 : ROWB == 64 ? LAYOUT_SW64 : LAYOUT_SW128;
  static constexpr int bytes(int rows) { return rows * D * 2; }
  // descriptor of the tile as an operand whose k runs along D
  __device__ static uint64_t desc_k(const void* base) { return umma_desc(smem_u32(base), 16, 8 * ROWB, LAYOUT); }
  // k-step kk (16 elements of D) of that operand, in a tile of `rows` rows
  __device__ static constexpr uint64_t kstep_k(int kk, int rows) {
    return static_cast<uint64_t>(((kk * 16 / PANEL) * rows * ROWB + (kk * 16 % PANEL) * 2) >> 4);
  }
  // descriptor of the tile as the B operand [D] x [rows] of a product over rows
  __device__ static uint64_t desc_mn(const void* base, int rows) {
    return umma_desc(smem_u32(base), rows * ROWB, 8 * ROWB, LAYOUT);
  }
  // k-step of 16 rows of that operand
  static constexpr uint64_t KSTEP_MN = (16 * ROWB) >> 4;
  // rows [row, row + rows) of (b, h) by TMA into `dst`
  __device__ static void load(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int row, int h, int b, int rows) {
#pragma unroll
    for (int p = 0; p < NP; ++p) tma_load_4d(dst + p * rows * ROWB, map, bar, p * PANEL, row, h, b);
  }
  // zero row r (swizzling permutes 16-byte pieces within a row of a panel only)
  __device__ static void zero_row(uint8_t* tile, int r, int rows) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int i = 0; i < ROWB / 16; ++i)
        *reinterpret_cast<uint4*>(tile + p * rows * ROWB + r * ROWB + 16 * i) = make_uint4(0, 0, 0, 0);
  }
};

}  // namespace flare
