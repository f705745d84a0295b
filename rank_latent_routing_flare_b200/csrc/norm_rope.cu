// Preparation of queries and keys: per-head RMS norm, gain and position
// rotation in one pass, and its gradients.  Per row x of one token and head:
//
//   r = rsqrt(mean(x^2) + eps),  y = x r g,  pairs (a, b) of y turned by t:
//   (a cos t - b sin t, a sin t + b cos t),  t = sum_i pos[n][i] freqs[i][p]
//
//   backward: u = the gradient turned back by t, w = u g,
//   dx = r (w - x r^2 mean(w x)),  dg = sum over rows of u x r
//
// Bound by HBM: every row is read once and written once (backward: two reads
// and one write).  A lane holds 8 elements (one 16-byte access), D / 8 lanes a
// row, so the row's sums are a few shuffles and nothing is staged.  The input
// usually is token-major (a slice of a projection) and the output head-major:
// a warp takes up to 64 / D heads of several tokens, so that both sides move
// in pieces of 128 bytes or more.  An angle is the same for every head of its
// token: a CTA first puts cos and sin of its tile's tokens into shared memory
// (position x frequency in fp64, reduced to a fraction of a turn there, so
// positions of 10^6 and more keep their angles; sine and cosine in fp32).
// Sums and products are fp32; results are rounded to bf16 once, at the store.
#include <algorithm>

#include "flare_internal.h"
#include "norm_rope.h"
#include "ptx.cuh"

namespace flare {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxBwdCtas = 3 * kNumSM;   // three resident CTAs per SM

// Heads a warp takes at once: 64 / D (128 bytes of a token-major row), or the
// largest power of two below that divides the head count.
__host__ __device__ inline int heads_per_item(int H, int D) {
  int ht = D >= 64 ? 1 : 64 / D;
  while (H % ht != 0) ht >>= 1;
  return ht;
}

// cos and sin of the tile's first `nvalid` tokens into cs[token][pair].
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, int b, int n0, int nvalid, float2* cs) {
  for (int i = threadIdx.x; i < nvalid * p.P; i += kThreads) {
    const int t = i / p.P, q = i - t * p.P, n = n0 + t;
    double a;
    if (p.pos_kind == 2) {
      const float* pos = static_cast<const float*>(p.pos) + (static_cast<long>(b) * p.N + n) * p.axes;
      a = 0.0;
      for (int k = 0; k < p.axes; ++k) a = fma(static_cast<double>(pos[k]), static_cast<double>(p.freqs[k * p.P + q]), a);
    } else {
      const int pos = p.pos_kind == 1 ? static_cast<const int*>(p.pos)[static_cast<long>(b) * p.N + n] : n;
      a = static_cast<double>(pos) * static_cast<double>(p.freqs[q]);
    }
    a *= 0.15915494309189533577;   // 1 / (2 pi): turns
    a -= rint(a);
    float sn, cn;
    sincospif(2.0f * static_cast<float>(a), &sn, &cn);
    cs[i] = make_float2(cn, sn);
  }
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 shfl4(const uint4& v, int src) {
  return make_uint4(__shfl_sync(~0u, v.x, src), __shfl_sync(~0u, v.y, src), __shfl_sync(~0u, v.z, src),
                    __shfl_sync(~0u, v.w, src));
}
__device__ __forceinline__ void load_gain(const float* g, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(g)), b = __ldg(reinterpret_cast<const float4*>(g) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// What a lane's 8 elements have to do with the rotation.
struct Turn {
  int src;      // lane that holds the other members of its pairs (half-split)
  int first;    // first pair of the lane's elements
  float sign;   // half-split: -1 where the elements are the pairs' first members, +1 second, 0 not rotated
  int npairs;   // interleaved: rotated pairs among the four
};
template <int D, bool IL>
__device__ __forceinline__ Turn lane_turn(int lane, int P) {
  constexpr int L = D / 8;
  const int l = lane % L;
  Turn t{lane, 0, 0.f, 0};
  if (IL) {
    t.first = 4 * l;
    t.npairs = max(0, min(4, P - 4 * l));
  } else {
    const int ph = P / 8;   // lanes that hold first members
    if (l < ph) {
      t.src = lane + ph;
      t.first = 8 * l;
      t.sign = -1.f;
    } else if (l < 2 * ph) {
      t.src = lane - ph;
      t.first = 8 * (l - ph);
      t.sign = 1.f;
    }
  }
  return t;
}
// v turned by the angles of its token (dir = 1) or back (dir = -1); other: the
// pairs' other members (half-split).
template <bool IL>
__device__ __forceinline__ void rotate(float (&v)[8], const float (&other)[8], const Turn& t, const float2* cs,
                                       float dir) {
  if (IL) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < t.npairs) {
        const float2 a = cs[t.first + i];
        const float s = dir * a.y, x = v[2 * i], y = v[2 * i + 1];
        v[2 * i] = fmaf(x, a.x, -y * s);
        v[2 * i + 1] = fmaf(x, s, y * a.x);
      }
  } else if (t.sign != 0.f) {
    const float4* c4 = reinterpret_cast<const float4*>(cs + t.first);
    const float d = dir * t.sign;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = c4[i];
      v[2 * i] = fmaf(v[2 * i], a.x, other[2 * i] * (d * a.y));
      v[2 * i + 1] = fmaf(v[2 * i + 1], a.z, other[2 * i + 1] * (d * a.w));
    }
  }
}

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Rows of one item: `tt` tokens of `ht` heads; lane -> (token, head, 8 elements).
struct Item {
  int ht, tt, h_in, t_in, l;
};
template <int D>
__device__ __forceinline__ Item lane_item(int H, int lane) {
  constexpr int L = D / 8;
  Item it;
  it.ht = heads_per_item(H, D);
  it.tt = (32 / L) / it.ht;
  it.l = lane % L;
  const int rr = lane / L;
  it.h_in = rr & (it.ht - 1);
  it.t_in = rr / it.ht;
  return it;
}

template <int D, bool IL>
__device__ __forceinline__ void fwd_side(const NormRopeParams& p, const NormRopeSide& s, int b, int n0, int ntok,
                                         int nvalid, const float2* cs) {
  constexpr int U = 4;   // items in flight per warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Item it = lane_item<D>(s.H, lane);
  const Turn turn = lane_turn<D, IL>(lane, p.P);
  const int ng = s.H / it.ht, ntg = (ntok + it.tt - 1) / it.tt, items = ng * ntg;
  const uint16_t* x0 = s.x + b * s.xs[0] + static_cast<long>(n0) * s.xs[2] + 8 * it.l;
  uint16_t* y0 = s.y + b * s.ys[0] + static_cast<long>(n0) * s.ys[2] + 8 * it.l;
  for (int i0 = warp; i0 < items; i0 += kWarps * U) {
    uint4 raw[U];
    int tok[U], head[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kWarps, tg = i / ng;
      tok[u] = i < items ? tg * it.tt + it.t_in : ntok;
      head[u] = (i - tg * ng) * it.ht + it.h_in;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (tok[u] < nvalid)
        raw[u] = *reinterpret_cast<const uint4*>(x0 + tok[u] * s.xs[2] + head[u] * s.xs[1]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * kWarps >= items) break;   // uniform over the warp
      float x[8], sq = 0.f;
      unpack8(raw[u], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
      const float r = rsqrtf(fmaf(row_sum<D>(sq), 1.0f / D, p.eps));
      float g[8], other[8];
      const float* gp = s.gain ? s.gain + (s.gain_per_head ? static_cast<long>(head[u]) * D : 0) : nullptr;
      if (gp) load_gain(gp + 8 * it.l, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= gp ? r * g[e] : r;
      if (!IL && p.P > 0) {
        unpack8(shfl4(raw[u], turn.src), other);
        if (gp) load_gain(gp + 8 * (turn.src % (D / 8)), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) other[e] *= gp ? r * g[e] : r;
      }
      if (tok[u] < nvalid && p.P > 0) rotate<IL>(x, other, turn, cs + tok[u] * p.P, 1.f);
      if (tok[u] < ntok)
        *reinterpret_cast<uint4*>(y0 + tok[u] * s.ys[2] + head[u] * s.ys[1]) =
            tok[u] < nvalid ? pack8(x) : make_uint4(0, 0, 0, 0);
    }
  }
}

__device__ __forceinline__ int valid_tokens(const NormRopeParams& p, int b, int n0, int ntok) {
  if (p.lengths == nullptr) return ntok;
  return max(0, min(ntok, p.lengths[b] - n0));
}

template <int D, bool IL>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_fwd_kernel(const NormRopeParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  float2* cs = reinterpret_cast<float2*>(smem);
  const int b = blockIdx.x / p.tiles_per_b, n0 = (blockIdx.x - b * p.tiles_per_b) * p.tile;
  const int ntok = min(p.tile, p.N - n0), nvalid = valid_tokens(p, b, n0, ntok);
  fill_angles(p, b, n0, nvalid, cs);
  __syncthreads();
  if (p.side[0].H) fwd_side<D, IL>(p, p.side[0], b, n0, ntok, nvalid, cs);
  if (p.side[1].H) fwd_side<D, IL>(p, p.side[1], b, n0, ntok, nvalid, cs);
}

// Backward.  A warp takes units: the token groups `part`, part + ts, ... of
// one group of heads, so that a lane's gain gradients stay in registers over
// them; each unit then adds to its own row of acc[ts][(Hq + Hk) D] in shared
// memory (no two warps share a row), and a CTA's rows are summed over its
// tiles in a fixed order.
template <int D, bool IL>
__device__ __forceinline__ void bwd_unit(const NormRopeParams& p, const NormRopeSide& s, int b, int n0, int ntok,
                                         int nvalid, const float2* cs, int group, int part, int ts, float* acc) {
  constexpr int U = 2;
  const int lane = threadIdx.x & 31;
  const Item it = lane_item<D>(s.H, lane);
  const Turn turn = lane_turn<D, IL>(lane, p.P);
  const int head = group * it.ht + it.h_in, ntg = (ntok + it.tt - 1) / it.tt;
  const uint16_t* x0 = s.x + b * s.xs[0] + head * s.xs[1] + static_cast<long>(n0) * s.xs[2] + 8 * it.l;
  const uint16_t* d0 = s.dy + b * s.ds[0] + head * s.ds[1] + static_cast<long>(n0) * s.ds[2] + 8 * it.l;
  uint16_t* y0 = s.y + b * s.ys[0] + head * s.ys[1] + static_cast<long>(n0) * s.ys[2] + 8 * it.l;
  float g[8], dg[8];
  if (s.gain) load_gain(s.gain + (s.gain_per_head ? static_cast<long>(head) * D : 0) + 8 * it.l, g);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (!s.gain) g[e] = 1.f;
    dg[e] = 0.f;
  }
  for (int tg0 = part; tg0 < ntg; tg0 += ts * U) {
    uint4 rx[U], rd[U];
    int tok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int tg = tg0 + u * ts;
      tok[u] = tg < ntg ? tg * it.tt + it.t_in : ntok;
      rx[u] = rd[u] = make_uint4(0, 0, 0, 0);
      if (tok[u] < nvalid) {
        rx[u] = *reinterpret_cast<const uint4*>(x0 + tok[u] * s.xs[2]);
        rd[u] = *reinterpret_cast<const uint4*>(d0 + tok[u] * s.ds[2]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (tg0 + u * ts >= ntg) break;   // uniform over the warp
      float x[8], v[8], other[8];
      unpack8(rx[u], x);
      unpack8(rd[u], v);
      if (!IL && p.P > 0) unpack8(shfl4(rd[u], turn.src), other);
      if (tok[u] < nvalid && p.P > 0) rotate<IL>(v, other, turn, cs + tok[u] * p.P, -1.f);
      float sq = 0.f, wx = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sq = fmaf(x[e], x[e], sq);
        wx = fmaf(v[e] * g[e], x[e], wx);
      }
      sq = row_sum<D>(sq);
      wx = row_sum<D>(wx);
      const float r = rsqrtf(fmaf(sq, 1.0f / D, p.eps));
      const float k = r * r * wx * (1.0f / D);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dg[e] = fmaf(v[e], x[e] * r, dg[e]);
        v[e] = r * fmaf(-x[e], k, v[e] * g[e]);
      }
      if (tok[u] < ntok)
        *reinterpret_cast<uint4*>(y0 + tok[u] * s.ys[2]) = tok[u] < nvalid ? pack8(v) : make_uint4(0, 0, 0, 0);
    }
  }
  if (s.dgain) {
    for (int o = it.ht * (D / 8); o < 32; o <<= 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) dg[e] += __shfl_xor_sync(~0u, dg[e], o);
    }
    if (it.t_in == 0) {
      float* a = acc + head * D + 8 * it.l;
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] += dg[e];
    }
  }
}

// Columns of a side's gain gradient in a CTA's partial row.
__host__ __device__ inline int gain_cols(const NormRopeSide& s, int D) {
  return s.dgain ? (s.gain_per_head ? s.H * D : D) : 0;
}

template <int D, bool IL>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_bwd_kernel(const NormRopeParams p, int ts, int acc_offset) {
  extern __shared__ __align__(16) uint8_t smem[];
  float2* cs = reinterpret_cast<float2*>(smem);
  float* acc = reinterpret_cast<float*>(smem + acc_offset);
  const int width = (p.side[0].H + p.side[1].H) * D;
  const bool gains = p.side[0].dgain || p.side[1].dgain;
  if (gains)
    for (int i = threadIdx.x; i < ts * width; i += kThreads) acc[i] = 0.f;
  const int ngq = p.side[0].H ? p.side[0].H / heads_per_item(p.side[0].H, D) : 0;
  const int ngk = p.side[1].H ? p.side[1].H / heads_per_item(p.side[1].H, D) : 0;
  const int ng = ngq + ngk;
  for (long tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x) {
    const int b = static_cast<int>(tile / p.tiles_per_b);
    const int n0 = static_cast<int>(tile - static_cast<long>(b) * p.tiles_per_b) * p.tile;
    const int ntok = min(p.tile, p.N - n0), nvalid = valid_tokens(p, b, n0, ntok);
    __syncthreads();   // the previous tile's angles are read
    fill_angles(p, b, n0, nvalid, cs);
    __syncthreads();
    for (int u = threadIdx.x >> 5; u < ng * ts; u += kWarps) {
      const int part = u / ng, group = u - part * ng;
      if (group < ngq)
        bwd_unit<D, IL>(p, p.side[0], b, n0, ntok, nvalid, cs, group, part, ts, acc + part * width);
      else
        bwd_unit<D, IL>(p, p.side[1], b, n0, ntok, nvalid, cs, group - ngq, part, ts,
                        acc + part * width + p.side[0].H * D);
    }
  }
  if (!gains) return;
  __syncthreads();
  const int cq = gain_cols(p.side[0], D), cols = cq + gain_cols(p.side[1], D);
  for (int c = threadIdx.x; c < cols; c += kThreads) {
    const int side = c < cq ? 0 : 1, k = c - (side ? cq : 0);
    const float* a = acc + (side ? p.side[0].H * D : 0) + k;
    const int heads = p.side[side].gain_per_head ? 1 : p.side[side].H;
    float sum = 0.f;
    for (int part = 0; part < ts; ++part)
      for (int h = 0; h < heads; ++h) sum += a[part * width + h * D];
    p.part[static_cast<long>(blockIdx.x) * cols + c] = sum;
  }
}

// Sum of the CTAs' partial rows, in a fixed order: 32 columns a block, the
// rows dealt to 32 warps, whose sums are added in order.
__global__ void __launch_bounds__(1024) gain_sum_kernel(const NormRopeParams p) {
  __shared__ float sh[32][33];
  const int cq = gain_cols(p.side[0], p.D), cols = cq + gain_cols(p.side[1], p.D);
  const int c = blockIdx.x * 32 + threadIdx.x;
  float sum = 0.f;
  if (c < cols)
    for (int i = threadIdx.y; i < p.ctas; i += 32) sum += p.part[static_cast<long>(i) * cols + c];
  sh[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
    float total = 0.f;
    for (int i = 0; i < 32; ++i) total += sh[i][threadIdx.x];
    (c < cq ? p.side[0].dgain : p.side[1].dgain)[c - (c < cq ? 0 : cq)] = total;
  }
}

template <typename F>
cudaError_t by_dim(int D, int interleaved, F&& f) {
  switch (D) {
    case 16: return interleaved ? f(std::integral_constant<int, 16>{}, std::true_type{}) : f(std::integral_constant<int, 16>{}, std::false_type{});
    case 32: return interleaved ? f(std::integral_constant<int, 32>{}, std::true_type{}) : f(std::integral_constant<int, 32>{}, std::false_type{});
    case 64: return interleaved ? f(std::integral_constant<int, 64>{}, std::true_type{}) : f(std::integral_constant<int, 64>{}, std::false_type{});
    case 128: return interleaved ? f(std::integral_constant<int, 128>{}, std::true_type{}) : f(std::integral_constant<int, 128>{}, std::false_type{});
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int norm_rope_bwd_ctas(long B, long N) { return static_cast<int>(std::min<long>(kMaxBwdCtas, B * N)); }

// Tokens per tile: enough that every thread has about 4 (backward: 16) pieces
// of 16 bytes, at most 32 KB of angles, and halved while the tiles would not
// give every SM two CTAs.
void norm_rope_plan(NormRopeParams* p, bool backward) {
  const long per_token = static_cast<long>(p->side[0].H + p->side[1].H) * (p->D / 8);
  long t = 32;
  while (t < 256 && t * per_token < (backward ? 16 : 4) * kThreads && 2 * t * p->P * 8 <= 32768) t *= 2;
  while (t > 1 && static_cast<long>(p->B) * ((p->N + t - 1) / t) < 2 * kNumSM) t /= 2;
  p->tile = static_cast<int>(t);
  p->tiles_per_b = static_cast<int>((p->N + t - 1) / t);
  p->n_tiles = static_cast<long>(p->B) * p->tiles_per_b;
  p->ctas = static_cast<int>(std::min<long>(kMaxBwdCtas, p->n_tiles));
}

cudaError_t launch_norm_rope_fwd(const NormRopeParams& p, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(p.tile) * p.P * 8;   // at most 32 KB
  return by_dim(p.D, p.interleaved, [&](auto d, auto il) {
    norm_rope_fwd_kernel<decltype(d)::value, decltype(il)::value>
        <<<static_cast<unsigned>(p.n_tiles), kThreads, smem, s>>>(p);
    return cudaGetLastError();
  });
}

cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, cudaStream_t s) {
  const int D = p.D, width = (p.side[0].H + p.side[1].H) * D;
  const int ng = (p.side[0].H ? p.side[0].H / heads_per_item(p.side[0].H, D) : 0) +
                 (p.side[1].H ? p.side[1].H / heads_per_item(p.side[1].H, D) : 0);
  // shares of a tile's tokens: as many as give the 8 warps equal numbers of
  // units, while the accumulators stay within 32 KB
  int ts = 1;
  while (ts < kWarps && (ng * ts) % kWarps != 0 && ng * ts < 8 * kWarps && 2 * ts * width * 4 <= 32768) ts *= 2;
  const bool gains = p.side[0].dgain || p.side[1].dgain;
  const int acc_offset = p.tile * p.P * 8;
  const size_t smem = acc_offset + (gains ? static_cast<size_t>(ts) * width * 4 : 0);
  const cudaError_t e = by_dim(D, p.interleaved, [&](auto d, auto il) {
    auto* kern = norm_rope_bwd_kernel<decltype(d)::value, decltype(il)::value>;
    if (smem > 48 * 1024) {
      const cudaError_t a = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (a != cudaSuccess) return a;
    }
    kern<<<static_cast<unsigned>(p.ctas), kThreads, smem, s>>>(p, ts, acc_offset);
    return cudaGetLastError();
  });
  if (e != cudaSuccess || !gains) return e;
  const int cols = gain_cols(p.side[0], D) + gain_cols(p.side[1], D);
  gain_sum_kernel<<<(cols + 31) / 32, dim3(32, 32), 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace flare
