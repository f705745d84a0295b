// Exact softmax attention of few query rows: single new tokens over a long
// cache.  A key head's query rows (its G query heads times Nq <= 16 rows)
// share every key and value, so K and V are read once and the kernel is bound
// by HBM.  The products are mma.sync m16n8k16 with the rows as columns, eight
// (NT = 1) or sixteen (NT = 2) of them: S^T = K Q^T, O^T += V^T P^T, far below the
// tensor pipe's rate, and little else to issue per key.
//
// Each warp streams chunks of 16 keys through a ring of its own in shared
// memory (16-byte cp.async, rows swizzled so that ldmatrix meets no bank
// conflict): what is in flight takes no registers, so that several CTAs of
// four warps share an SM and one's beginning and end run under the others'
// loads.  K's fragments come from ldmatrix, V's from its transposing form; the
// weights turn from a sum's layout into an operand's by movmatrix.  Rows keep a
// running reference and sum as in the tiled kernel.  The keys are split over
// CTAs, within a CTA over its warps, which join in shared memory; up to eight
// splits are a cluster and join there too.
//
// D = 128, 8 key heads of 4 query heads, ragged caches: 16 of up to 32768 keys 194
// us with the join, 6.9 TB/s; 64 of up to 1024 31 us, 5.1.  (Chunks in
// registers, one CTA of 8 warps an SM, rows as the products' 16 rows: 258 and 96.
// As here but for the rows: 216 and 43, half of the issue slots taken.)
#include <climits>
#include <tuple>
#include <type_traits>

#include "attn_common.cuh"
#include "ops_internal.h"

namespace flare {
namespace {

constexpr int kStepWarps = 4, kChunk = 16;

struct StepParams {
  AttnParams a;
  AttnSide q, k, v;
};

template <int D>
struct StepCfg {
  static constexpr int U = D / 8;                       // 16-byte units of a row
  static constexpr int CHUNK_B = kChunk * D * 2;        // K's or V's part of a chunk
  static constexpr int STAGES = D == 128 ? 2 : D == 64 ? 3 : 4;
  static constexpr int CTAS = D == 128 ? 3 : D == 64 ? 4 : 6;
  static constexpr int RING_B = kStepWarps * STAGES * 2 * CHUNK_B;
  // 16-byte unit u of row r of a chunk: eight rows of the same unit, and eight units of a row, lie in different banks
  __device__ static constexpr int swizzle(int r) { return U >= 8 ? r & 7 : U == 4 ? r >> 1 & 3 : r >> 2 & 1; }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {   // zeros if not ok
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 x 8 values, row g of lanes (g, 0 .. 3), to column g.
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

// Copies of a chunk's rows of K and V, zeros from key `end` on and for V's before `beg`.
template <int D>
__device__ __forceinline__ void load_chunk(uint32_t dst, const StepParams& p, const BatchMask& m, const uint16_t* kb,
                                           const uint16_t* vb, int key0, int beg, int end) {
  using C = StepCfg<D>;
  constexpr int ROWS = 32 / C::U, N = kChunk / ROWS;   // rows a warp copies at once
  const int lane = threadIdx.x & 31, r0 = lane / C::U, u = lane % C::U;
  const uint32_t at0 = 2 * D * r0 + 16 * (u ^ C::swizzle(r0));
  auto at = [&](int i) { return dst + (at0 ^ 16 * C::swizzle(i * ROWS)) + 2 * D * ROWS * i; };
  const uint16_t *k = kb + static_cast<long>(key0 + r0) * p.k.sn + 8 * u, *v = vb + static_cast<long>(key0 + r0) * p.v.sn + 8 * u;
  if (key0 >= beg && key0 + kChunk <= end && !m.doc) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      copy16(at(i), k);
      copy16(at(i) + C::CHUNK_B, v);
      k += ROWS * p.k.sn;
      v += ROWS * p.v.sn;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int key = key0 + r0 + i * ROWS;
    bool ok = key < end;
    copy16(at(i), ok ? k + i * ROWS * p.k.sn : kb, ok);
    ok = ok && key >= beg;   // a weight of 0 does not erase a NaN: what no row sees is not read
    if (m.doc && ok) {
      const int2 d = m.doc[key];
      ok = d.x != d.y;
    }
    copy16(at(i) + C::CHUNK_B, ok ? v + i * ROWS * p.v.sn : vb, ok);
  }
}

// CAP: capped scores; without, the tanh's coefficients take no registers.
template <int D, bool CAP, int NT>
__global__ void __launch_bounds__(kStepWarps * 32, StepCfg<D>::CTAS) attn_step_kernel(const StepParams p) {
  using C = StepCfg<D>;
  extern __shared__ uint8_t sh_raw[];   // the warps' rings; behind the loop the join's data
  uint8_t* sh = sh_raw + (256 - smem_u32(sh_raw) % 256) % 256;   // rows on multiples of their size
  const AttnParams& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x % a.splits, bk = blockIdx.x / a.splits, b = bk / a.Hk, hk = bk % a.Hk;
  const int rows = a.G * a.mask.Nq;
  const BatchMask mask = batch_mask(a.mask, b);

  // the keys that any row sees, rounded to chunks and dealt to the splits
  int seen = 0, lo = 0, hi = 0;
  const int last_row = min(a.mask.Nq, mask.qlen) - 1;
  if (blockIdx.x == 0 && threadIdx.x < 4) a.err[threadIdx.x] = 0u;   // nothing here can wait in vain
  if (last_row >= 0) {
    seen = row_interval(mask, 0).x;
    lo = seen / kChunk * kChunk;
    hi = row_interval(mask, last_row).y;
  }
  const int chunks = hi > lo ? (hi - lo + kChunk - 1) / kChunk : 0;
  const int per = (chunks + a.splits - 1) / a.splits;
  const int c_end = min(chunks, (split + 1) * per);

  const uint16_t* kb = p.k.p + b * p.k.sb + hk * p.k.sh;
  const uint16_t* vb = p.v.p + b * p.v.sb + hk * p.v.sh;
  const uint32_t ring = smem_u32(sh) + warp * C::STAGES * 2 * C::CHUNK_B;
  const int c_beg = split * per + warp;
  auto load = [&](int n) {   // the warp's chunk n
    const int c = c_beg + n * kStepWarps;
    if (c < c_end) load_chunk<D>(ring + n % C::STAGES * 2 * C::CHUNK_B, p, mask, kb, vb, lo + c * kChunk, seen, hi);
    copies_end();
  };
#pragma unroll
  for (int n = 0; n < C::STAGES - 1; ++n) load(n);

  // this lane's rows 8 v + 2 t + u: r = i G + head
  int2 iv[NT][2];
  int pos[NT][2];
  float slope2[NT][2];
  int all_lo = 0, all_hi = INT_MAX;   // keys that every row sees
  __shared__ uint2 sm_q[D / 16][NT][32];   // Q's operand fragments, the same for every warp: read per chunk, they hold no registers
  const ScoreOps ops(a.scale, a.cap, true);
#pragma unroll
  for (int v = 0; v < NT; ++v) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = 8 * v + 2 * t + u, i = r / a.G, h = hk * a.G + r % a.G;
      const bool have = r < rows;
      iv[v][u] = have ? row_interval(mask, i) : make_int2(0, INT_MAX);   // (what is no row may see anything)
      pos[v][u] = bias_position(mask, have ? i : 0, iv[v][u]);
      slope2[v][u] = have && a.slopes ? a.slopes[h] * kLog2e : 0.f;
      all_lo = max(all_lo, iv[v][u].x);
      all_hi = min(all_hi, iv[v][u].y);
    }
    const int r = 8 * v + g, i = r / a.G, h = hk * a.G + r % a.G;
    const uint16_t* q = p.q.p + b * p.q.sb + h * p.q.sh + static_cast<long>(i) * p.q.sn + 2 * t;
    for (int k = warp; k < D / 16; k += kStepWarps)
      sm_q[k][v][lane] = r < rows ? make_uint2(*reinterpret_cast<const uint32_t*>(q + 16 * k),
                                               *reinterpret_cast<const uint32_t*>(q + 16 * k + 8))
                                  : make_uint2(0u, 0u);
  }
#pragma unroll
  for (int x = 1; x < 4; x *= 2) {
    all_lo = max(all_lo, __shfl_xor_sync(~0u, all_lo, x));
    all_hi = min(all_hi, __shfl_xor_sync(~0u, all_hi, x));
  }
  __syncthreads();

  float o[D / 16][NT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int v = 0; v < NT; ++v) {
    m[v][0] = m[v][1] = -INFINITY;
    l[v][0] = l[v][1] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[j][v][k] = 0.f;
  }
  // where this lane's rows lie in ldmatrix: keys 0-7, 8-15 by the first (K) or the second (V) half of 16 columns, and so on
  const int rk = lane & 15, rv = (lane >> 4) * 8 + (lane & 7);
  const uint32_t at_k = 2 * D * rk + 16 * ((lane >> 4) ^ C::swizzle(rk));
  const uint32_t at_v = C::CHUNK_B + 2 * D * rv + 16 * ((lane >> 3 & 1) ^ C::swizzle(rv));

  auto compute = [&](uint32_t chunk, int key0) {
    float s[NT][4];
#pragma unroll
    for (int v = 0; v < NT; ++v)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[v][k] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t kf[4];
      ldmatrix(kf, (chunk + at_k) ^ 32 * k);
#pragma unroll
      for (int v = 0; v < NT; ++v) {
        uint32_t q[2];
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(q[0]), "=r"(q[1]) : "r"(smem_u32(&sm_q[k][v][lane])));
        mma16816(s[v], kf, q[0], q[1]);
      }
    }
    if (CAP) {
      float top = 0.f;
#pragma unroll
      for (int v = 0; v < NT; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmaxf(top, fabsf(s[v][k]));
      const bool small = __all_sync(~0u, ops.small(top));
#pragma unroll
      for (int v = 0; v < NT; ++v) {
        if (small) {
          f2_unpack(ops.poly(f2_pack(s[v][0], s[v][1]), f2_dup(0.f)), s[v][0], s[v][1]);
          f2_unpack(ops.poly(f2_pack(s[v][2], s[v][3]), f2_dup(0.f)), s[v][2], s[v][3]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) s[v][k] = ops.capped(s[v][k]);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < NT; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[v][k] *= ops.c2;
    }
    if (a.slopes) {
#pragma unroll
      for (int v = 0; v < NT; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          s[v][k] = fmaf(-slope2[v][k & 1], fabsf(static_cast<float>(pos[v][k & 1] - (key0 + g + 8 * (k >> 1)))), s[v][k]);
    }
    if (key0 < all_lo || key0 + kChunk > all_hi) {
#pragma unroll
      for (int v = 0; v < NT; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = key0 + g + 8 * (k >> 1);
          if (key < iv[v][k & 1].x || key >= iv[v][k & 1].y) s[v][k] = -INFINITY;
        }
    }
    bool grown = false;
#pragma unroll
    for (int v = 0; v < NT; ++v)
#pragma unroll
      for (int u = 0; u < 2; ++u) grown |= fmaxf(s[v][u], s[v][2 + u]) > m[v][u] + 8.f;
    if (__any_sync(~0u, grown)) {
#pragma unroll
      for (int v = 0; v < NT; ++v) {
        float f[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float mx = fmaxf(s[v][u], s[v][2 + u]);
#pragma unroll
          for (int x = 4; x < 32; x *= 2) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, x));
          const float m_new = fmaxf(m[v][u], mx);
          f[u] = m[v][u] == -INFINITY ? 0.f : ex2_mufu(m[v][u] - m_new);
          m[v][u] = m_new;
          l[v][u] *= f[u];
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[j][v][k] *= f[k & 1];
      }
    }
    uint32_t pf[NT][2];
#pragma unroll
    for (int v = 0; v < NT; ++v) {
      const float b0 = m[v][0] == -INFINITY ? 0.f : m[v][0], b1 = m[v][1] == -INFINITY ? 0.f : m[v][1];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float p0 = ex2_mufu(s[v][2 * n] - b0), p1 = ex2_mufu(s[v][2 * n + 1] - b1);
        l[v][0] += p0;
        l[v][1] += p1;
        pf[v][n] = transposed(pack_bf16x2(p0, p1));
      }
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint32_t vf[4];
      ldmatrix_trans(vf, (chunk + at_v) ^ 32 * j);
#pragma unroll
      for (int v = 0; v < NT; ++v) mma16816(o[j][v], vf, pf[v][0], pf[v][1]);
    }
  };
  for (int n = 0; c_beg + n * kStepWarps < c_end; ++n) {
    copies_wait<C::STAGES - 2>();
    __syncwarp();              // every lane's copies of chunk n are there, and chunk n - 1 has been read
    load(n + C::STAGES - 1);
    compute(ring + n % C::STAGES * 2 * C::CHUNK_B, lo + (c_beg + n * kStepWarps) * kChunk);
  }
  copies_wait<0>();
  __syncthreads();             // the join's data go over the rings

  // join the warps: row statistics, then the outputs
  float* sm_ml = reinterpret_cast<float*>(sh);
  float* sm_o = sm_ml + 2 * kStepWarps * rows;
  // a cluster's partial outputs and log2 sums, behind the warps'
  float* sm_part = sm_o + kStepWarps * rows * D;
  float* sm_lse = sm_part + rows * (D + 4);
  const bool in_cluster = a.splits > 1 && a.splits <= kAttnClusterSplits;
#pragma unroll
  for (int v = 0; v < NT; ++v)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int x = 4; x < 32; x *= 2) l[v][u] += __shfl_xor_sync(~0u, l[v][u], x);
      const int r = 8 * v + 2 * t + u;
      if (r < rows) {
        if (g == 0) {
          sm_ml[2 * (warp * rows + r)] = m[v][u];
          sm_ml[2 * (warp * rows + r) + 1] = l[v][u];
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          float* d = sm_o + (warp * rows + r) * D + 16 * j + g;
          d[0] = o[j][v][u];
          d[8] = o[j][v][2 + u];
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
constexpr int join_smem(int rows, int D) { return 4 * rows * (kStepWarps * (D + 2) + D + 5); }

}  // namespace

int attn_step_ctas(int D) {
  return D == 128 ? StepCfg<128>::CTAS : D == 64 ? StepCfg<64>::CTAS : D == 32 ? StepCfg<32>::CTAS : StepCfg<16>::CTAS;
}

cudaError_t launch_attn_step(const AttnParams& p, const AttnSide& q, const AttnSide& k, const AttnSide& v,
                             cudaStream_t s) {
  const StepParams sp{p, q, k, v};
  const dim3 grid(static_cast<unsigned>(static_cast<long>(p.splits) * p.B * p.Hk));
  auto go = [&](auto d, auto cap, auto nt) {
    constexpr int D = decltype(d)::value;
    using C = StepCfg<D>;
    static_assert(join_smem(kAttnStepRows, D) <= C::RING_B, "the join's data fit over the rings");
    static_assert(C::CTAS * (C::RING_B + 256 + 32 * D + 1024) <= 228 * 1024, "shared memory");
    auto* kern = attn_step_kernel<D, decltype(cap)::value, decltype(nt)::value>;
    constexpr int smem = C::RING_B + 256;
    const cudaError_t e = allow_smem<std::tuple<C, decltype(cap), decltype(nt)>>(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_splits(kern, grid, kStepWarps * 32, smem, s, dim3(p.splits, 1, 1), p.splits, sp);
  };
  auto by_rows = [&](auto d, auto cap) {
    return p.G * p.mask.Nq <= 8 ? go(d, cap, std::integral_constant<int, 1>{}) : go(d, cap, std::integral_constant<int, 2>{});
  };
  auto by_cap = [&](auto d) { return p.cap > 0.f ? by_rows(d, std::true_type{}) : by_rows(d, std::false_type{}); };
  switch (p.D) {
    case 16: return by_cap(std::integral_constant<int, 16>{});
    case 32: return by_cap(std::integral_constant<int, 32>{});
    case 64: return by_cap(std::integral_constant<int, 64>{});
    case 128: return by_cap(std::integral_constant<int, 128>{});
  }
  return cudaErrorInvalidValue;
}

}  // namespace flare
