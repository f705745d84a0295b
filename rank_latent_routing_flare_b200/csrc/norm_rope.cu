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
// a warp takes a group of up to 64 / D heads of several tokens, so that both
// sides move in pieces of 128 bytes or more.  It stays with its group: gains
// and, in the backward, the gains' gradients are registers over all of its
// tokens.  An angle is the same for every head of its token: the CTA first
// puts cos and sin of a tile's tokens into shared memory (position x
// frequency in fp64, reduced to a fraction of a turn there, so positions of
// 10^6 and more keep their angles; sine and cosine in fp32).
// Sums and products are fp32, in paired instructions; results are rounded to
// bf16 once, at the store.
#include <algorithm>

#include "flare_internal.h"
#include "norm_rope.h"
#include "ptx.cuh"

namespace flare {
namespace {

constexpr int kMaxWarps = 8;
constexpr int kWarpsPerSM = 24;   // resident at 80 registers a thread
constexpr int kRedCols = 128;     // columns of a group: ht * D

// Heads of a group: 64 / D (128 bytes of a token-major row), or the largest
// power of two below that divides the head count.
__host__ __device__ inline int heads_per_group(int H, int D) {
  int ht = D >= 64 ? 1 : 64 / D;
  while (H % ht != 0) ht >>= 1;
  return ht;
}
__host__ __device__ inline int groups_of(int H, int D) { return H ? H / heads_per_group(H, D) : 0; }

// Columns of the angle table: the rotated pairs, or with interleaved pairs
// all D / 2 of them (an angle of 0 for those that are not rotated).
template <int D, bool IL>
__device__ __forceinline__ int table_width(int P) { return IL ? D / 2 : P; }

// cos and sin of the tile's first `nvalid` tokens: cs[token][cos W | sin W].
template <int D, bool IL>
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, int b, int n0, int nvalid, float* cs) {
  const int W = table_width<D, IL>(p.P);
  const int bits = W <= 1 ? 0 : 32 - __clz(W - 1);          // a thread keeps one pair
  const int q = threadIdx.x & ((1 << bits) - 1), step = blockDim.x >> bits, t0 = threadIdx.x >> bits;
  if (q >= W || t0 >= step) return;
  double f[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    f[k] = k < p.axes && q < p.P ? static_cast<double>(p.freqs[k * p.P + q]) * 0.15915494309189533577 : 0.0;   // turns
  for (int t = t0; t < nvalid; t += step) {
    const int n = n0 + t;
    double a;
    if (p.pos_kind == 2) {
      const float* pos = static_cast<const float*>(p.pos) + (static_cast<long>(b) * p.N + n) * p.axes;
      a = static_cast<double>(pos[0]) * f[0];
#pragma unroll
      for (int k = 1; k < 4; ++k)
        if (k < p.axes) a = fma(static_cast<double>(pos[k]), f[k], a);
    } else {
      a = static_cast<double>(p.pos_kind == 1 ? static_cast<const int*>(p.pos)[static_cast<long>(b) * p.N + n] : n) * f[0];
    }
    a -= rint(a);
    float sn, cn;
    sincospif(2.0f * static_cast<float>(a), &sn, &cn);
    cs[t * 2 * W + q] = cn;
    cs[t * 2 * W + W + q] = sn;
  }
}

// 8 elements of a row as four fp32 pairs.
struct Vec8 {
  uint64_t v[4];
};
__device__ __forceinline__ Vec8 unpack(const uint4& r) {
  return Vec8{{f2_pack(bf16_lo(r.x), bf16_hi(r.x)), f2_pack(bf16_lo(r.y), bf16_hi(r.y)),
               f2_pack(bf16_lo(r.z), bf16_hi(r.z)), f2_pack(bf16_lo(r.w), bf16_hi(r.w))}};
}
__device__ __forceinline__ uint32_t round_pair(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint4 pack(const Vec8& x) {
  return make_uint4(round_pair(x.v[0]), round_pair(x.v[1]), round_pair(x.v[2]), round_pair(x.v[3]));
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) { return f2_fma(a, b, f2_pack(-0.f, -0.f)); }
__device__ __forceinline__ uint64_t f2_dup(float a) { return f2_pack(a, a); }
__device__ __forceinline__ Vec8 load_gain(const float* g) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(g)), b = __ldg(reinterpret_cast<const float4*>(g) + 1);
  return Vec8{{f2_pack(a.x, a.y), f2_pack(a.z, a.w), f2_pack(b.x, b.y), f2_pack(b.z, b.w)}};
}
__device__ __forceinline__ float sum8(const Vec8& a, const Vec8& b) {   // <a, b>
  uint64_t s = f2_mul(a.v[0], b.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = f2_fma(a.v[i], b.v[i], s);
  float lo, hi;
  f2_unpack(s, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ uint4 shfl4(const uint4& v, int src) {
  return make_uint4(__shfl_sync(~0u, v.x, src), __shfl_sync(~0u, v.y, src), __shfl_sync(~0u, v.z, src),
                    __shfl_sync(~0u, v.w, src));
}
template <int D>
__device__ __forceinline__ float row_sum(float v) {   // over the D / 8 lanes of a row
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// The turn of a lane's 8 elements.  Half-split pairs: y = v cos + o sin, o the
// pairs' other members (of lane src), already signed: -o for the first
// members of a forward turn, +o for the second.  Interleaved pairs lie within
// the lane; dir = 1 forward, -1 back.
struct Turn {
  int src, first;
  bool turned;
  float sign;
};
template <int D, bool IL>
__device__ __forceinline__ Turn lane_turn(int lane, int P) {
  const int l = lane % (D / 8);
  if (IL) return Turn{lane, 4 * l, 4 * l < P, 1.f};
  const int ph = P / 8;
  if (l < ph) return Turn{lane + ph, 8 * l, true, -1.f};
  if (l < 2 * ph) return Turn{lane - ph, 8 * (l - ph), true, 1.f};
  return Turn{lane, 0, false, 0.f};
}
template <bool IL>
__device__ __forceinline__ void rotate(Vec8& v, const Vec8& o, const Turn& t, const float* cs, int W, float dir) {
  const float4* c4 = reinterpret_cast<const float4*>(cs + t.first);
  const float4* s4 = reinterpret_cast<const float4*>(cs + W + t.first);
  if (IL) {
    const float4 c = c4[0], s = s4[0];
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      f2_unpack(v.v[i], a, b);
      const float sn = dir * ss[i];
      v.v[i] = f2_fma(f2_pack(-b, a), f2_dup(sn), f2_mul(v.v[i], f2_dup(cc[i])));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c = c4[i], s = s4[i];
      v.v[2 * i] = f2_fma(o.v[2 * i], f2_pack(s.x, s.y), f2_mul(v.v[2 * i], f2_pack(c.x, c.y)));
      v.v[2 * i + 1] = f2_fma(o.v[2 * i + 1], f2_pack(s.z, s.w), f2_mul(v.v[2 * i + 1], f2_pack(c.z, c.w)));
    }
  }
}

// A lane's place in its warp's group: token t_in of tt, head h_in of ht, and
// 8 elements from 8 l.
template <int D>
struct Place {
  int ht, tt, h_in, t_in, l;
  __device__ __forceinline__ Place(int H, int lane) {
    constexpr int L = D / 8;
    ht = heads_per_group(H, D);
    tt = (32 / L) / ht;
    l = lane % L;
    const int rr = lane / L;
    h_in = rr & (ht - 1);
    t_in = rr / ht;
  }
};

__device__ __forceinline__ int valid_tokens(const NormRopeParams& p, int b, int n0, int ntok) {
  if (p.lengths == nullptr) return ntok;
  return max(0, min(ntok, p.lengths[b] - n0));
}

// This warp's group of the CTA and its share of a tile's tokens.
struct Unit {
  int group, part, side;   // group within its side; side -1: none
};
__device__ __forceinline__ Unit warp_unit(const NormRopeParams& p) {
  const int warp = threadIdx.x >> 5, part = warp / p.cta_groups;
  const int g = static_cast<int>(blockIdx.x % p.ctas_y) * p.cta_groups + warp - part * p.cta_groups;
  const int nq = groups_of(p.side[0].H, p.D);
  return g >= p.groups ? Unit{0, part, -1} : g < nq ? Unit{g, part, 0} : Unit{g - nq, part, 1};
}

template <int D, bool IL>
__global__ void __launch_bounds__(32 * kMaxWarps, kWarpsPerSM / kMaxWarps) norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p) {
  extern __shared__ __align__(16) float cs[];
  constexpr int U = 4;   // rows in flight per lane
  const int lane = threadIdx.x & 31;
  const long tile = blockIdx.x / p.ctas_y;
  const int b = static_cast<int>(tile / p.tiles_per_b);
  const int n0 = static_cast<int>(tile - static_cast<long>(b) * p.tiles_per_b) * p.tile;
  const int ntok = min(p.tile, p.N - n0), nvalid = valid_tokens(p, b, n0, ntok);
  const Unit unit = warp_unit(p);
  if (p.P > 0) {
    fill_angles<D, IL>(p, b, n0, nvalid, cs);
    __syncthreads();
  }
  if (unit.side < 0) return;
  const NormRopeSide& s = p.side[unit.side];
  const Place<D> at(s.H, lane);
  const Turn turn = lane_turn<D, IL>(lane, p.P);
  const int W = table_width<D, IL>(p.P), head = unit.group * at.ht + at.h_in;
  const uint16_t* x0 = s.x + b * s.xs[0] + head * s.xs[1] + static_cast<long>(n0) * s.xs[2] + 8 * at.l;
  uint16_t* y0 = s.y + b * s.ys[0] + head * s.ys[1] + static_cast<long>(n0) * s.ys[2] + 8 * at.l;
  // the gain, and for half-split pairs the signed gain of the other members
  Vec8 g, go;
  const float* gp = s.gain + (s.gain_per_head ? static_cast<long>(head) * D : 0);
  if (s.gain) g = load_gain(gp + 8 * at.l);
  if (s.gain && !IL) go = load_gain(gp + 8 * (turn.src % (D / 8)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!s.gain) g.v[i] = go.v[i] = f2_dup(1.f);
    if (!IL) go.v[i] = f2_mul(go.v[i], f2_dup(turn.sign));
  }
  const int step = p.parts * at.tt;   // tokens between a lane's rows
  for (int t0 = unit.part * at.tt; t0 < ntok; t0 += U * step) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * step + at.t_in;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (t < nvalid) raw[u] = *reinterpret_cast<const uint4*>(x0 + t * s.xs[2]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t0 + u * step >= ntok) break;   // uniform over the warp
      const int t = t0 + u * step + at.t_in;
      Vec8 x = unpack(raw[u]), o;
      const uint64_t r = f2_dup(rsqrtf(fmaf(row_sum<D>(sum8(x, x)), 1.0f / D, p.eps)));
#pragma unroll
      for (int i = 0; i < 4; ++i) x.v[i] = f2_mul(x.v[i], f2_mul(g.v[i], r));
      if (!IL && p.P > 0) {
        o = unpack(shfl4(raw[u], turn.src));
#pragma unroll
        for (int i = 0; i < 4; ++i) o.v[i] = f2_mul(o.v[i], f2_mul(go.v[i], r));
      }
      if (turn.turned && t < nvalid) rotate<IL>(x, o, turn, cs + t * 2 * W, W, 1.f);
      if (t < ntok) *reinterpret_cast<uint4*>(y0 + t * s.ys[2]) = t < nvalid ? pack(x) : make_uint4(0, 0, 0, 0);
    }
  }
}

// Columns of a side's gain gradient in a CTA's partial row.
__host__ __device__ inline int gain_cols(const NormRopeSide& s, int D) {
  return s.dgain ? (s.gain_per_head ? s.H * D : D) : 0;
}

template <int D, bool IL>
__global__ void __launch_bounds__(32 * kMaxWarps, kWarpsPerSM / kMaxWarps) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  extern __shared__ __align__(16) float cs[];
  __shared__ float red[kMaxWarps][kRedCols];
  constexpr int U = 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int range = static_cast<int>(blockIdx.x / p.ctas_y);
  const Unit unit = warp_unit(p);
  const NormRopeSide& s = p.side[max(unit.side, 0)];
  const Place<D> at(max(s.H, 1), lane);
  const Turn turn = lane_turn<D, IL>(lane, p.P);
  const int W = table_width<D, IL>(p.P), head = unit.group * at.ht + at.h_in;
  Vec8 g, dg;
  if (s.gain) g = load_gain(s.gain + (s.gain_per_head ? static_cast<long>(head) * D : 0) + 8 * at.l);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!s.gain) g.v[i] = f2_dup(1.f);
    dg.v[i] = f2_dup(0.f);
  }
  const uint64_t back = f2_dup(-turn.sign);
  for (long tile = range; tile < p.n_tiles; tile += p.ranges) {
    const int b = static_cast<int>(tile / p.tiles_per_b);
    const int n0 = static_cast<int>(tile - static_cast<long>(b) * p.tiles_per_b) * p.tile;
    const int ntok = min(p.tile, p.N - n0), nvalid = valid_tokens(p, b, n0, ntok);
    if (p.P > 0) {
      __syncthreads();   // the previous tile's angles are read
      fill_angles<D, IL>(p, b, n0, nvalid, cs);
      __syncthreads();
    }
    if (unit.side < 0) continue;
    const uint16_t* x0 = s.x + b * s.xs[0] + head * s.xs[1] + static_cast<long>(n0) * s.xs[2] + 8 * at.l;
    const uint16_t* d0 = s.dy + b * s.ds[0] + head * s.ds[1] + static_cast<long>(n0) * s.ds[2] + 8 * at.l;
    uint16_t* y0 = s.y + b * s.ys[0] + head * s.ys[1] + static_cast<long>(n0) * s.ys[2] + 8 * at.l;
    const int step = p.parts * at.tt;
    for (int t0 = unit.part * at.tt; t0 < ntok; t0 += U * step) {
      uint4 rx[U], rd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * step + at.t_in;
        rx[u] = rd[u] = make_uint4(0, 0, 0, 0);
        if (t < nvalid) {
          rx[u] = *reinterpret_cast<const uint4*>(x0 + t * s.xs[2]);
          rd[u] = *reinterpret_cast<const uint4*>(d0 + t * s.ds[2]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t0 + u * step >= ntok) break;   // uniform over the warp
        const int t = t0 + u * step + at.t_in;
        Vec8 x = unpack(rx[u]), v = unpack(rd[u]), o;
        if (!IL && p.P > 0) {
          o = unpack(shfl4(rd[u], turn.src));
#pragma unroll
          for (int i = 0; i < 4; ++i) o.v[i] = f2_mul(o.v[i], back);
        }
        if (turn.turned && t < nvalid) rotate<IL>(v, o, turn, cs + t * 2 * W, W, -1.f);
        const float sq = row_sum<D>(sum8(x, x));
        Vec8 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w.v[i] = f2_mul(v.v[i], g.v[i]);
        const float wx = row_sum<D>(sum8(w, x));
        const float r = rsqrtf(fmaf(sq, 1.0f / D, p.eps));
        const uint64_t r2 = f2_dup(r), k2 = f2_dup(-r * r * wx * (1.0f / D));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dg.v[i] = f2_fma(v.v[i], f2_mul(x.v[i], r2), dg.v[i]);
          w.v[i] = f2_mul(r2, f2_fma(x.v[i], k2, w.v[i]));
        }
        if (t < ntok) *reinterpret_cast<uint4*>(y0 + t * s.ys[2]) = t < nvalid ? pack(w) : make_uint4(0, 0, 0, 0);
      }
    }
  }
  const int cq = gain_cols(p.side[0], D), cols = cq + gain_cols(p.side[1], D);
  if (cols == 0) return;
  // the CTA's partial row: lanes of one head, then the warps, in a fixed order
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(dg.v[i], f[2 * i], f[2 * i + 1]);
  for (int o = at.ht * (D / 8); o < 32; o <<= 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += __shfl_xor_sync(~0u, f[e], o);
  }
  if (at.t_in == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) red[warp][at.h_in * D + 8 * at.l + e] = f[e];
  }
  __syncthreads();
  float* row = p.part + static_cast<long>(blockIdx.x) * cols;
  const int nq = groups_of(p.side[0].H, D), g0 = static_cast<int>(blockIdx.x % p.ctas_y) * p.cta_groups;
  for (int side = 0; side < 2; ++side) {
    const NormRopeSide& sd = p.side[side];
    if (!sd.dgain) continue;
    const int ht = heads_per_group(sd.H, D), base = side ? nq : 0;
    // this CTA's groups of the side: warps [w0, w1) of every share
    const int w0 = max(base - g0, 0), w1 = min(min(base + sd.H / ht, p.groups) - g0, p.cta_groups);
    float* out = row + (side ? cq : 0);
    if (sd.gain_per_head) {
      for (int c = threadIdx.x; c < max(w1 - w0, 0) * ht * D; c += blockDim.x) {
        const int w = w0 + c / (ht * D), k = c % (ht * D);
        float sum = 0.f;
        for (int part = 0; part < p.parts; ++part) sum += red[part * p.cta_groups + w][k];
        out[(g0 + w - base) * ht * D + k] = sum;
      }
    } else if (w0 < w1) {
      for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float sum = 0.f;
        for (int part = 0; part < p.parts; ++part)
          for (int w = w0; w < w1; ++w)
            for (int h = 0; h < ht; ++h) sum += red[part * p.cta_groups + w][h * D + d];
        out[d] = sum;
      }
    }
  }
}

// Sum of the CTAs' partial rows, in a fixed order: 32 columns a block, the
// rows that hold the column dealt to 32 warps, whose sums are added in order.
__global__ void __launch_bounds__(1024) gain_sum_kernel(const __grid_constant__ NormRopeParams p) {
  __shared__ float sh[32][33];
  const int cq = gain_cols(p.side[0], p.D), cols = cq + gain_cols(p.side[1], p.D);
  const int c = blockIdx.x * 32 + threadIdx.x;
  const int side = c < cq ? 0 : 1, k = c - (side ? cq : 0);
  const NormRopeSide& s = p.side[side];
  float sum = 0.f;
  if (c < cols) {
    const int ht = heads_per_group(s.H, p.D), base = side ? groups_of(p.side[0].H, p.D) : 0;
    // CTAs of a range whose groups hold the column: one, or all with a group of the side
    const int first = s.gain_per_head ? base + k / (ht * p.D) : base, last = s.gain_per_head ? first : base + s.H / ht - 1;
    const int y0 = first / p.cta_groups, ny = last / p.cta_groups - y0 + 1;
    for (int i = threadIdx.y; i < p.ranges * ny; i += 32)
      sum += p.part[(static_cast<long>(i / ny) * p.ctas_y + y0 + i % ny) * cols + c];
  }
  sh[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
    float total = 0.f;
    for (int i = 0; i < 32; ++i) total += sh[i][threadIdx.x];
    s.dgain[k] = total;
  }
}

template <typename F>
cudaError_t by_dim(int D, int interleaved, F&& f) {
  auto go = [&](auto d) { return interleaved ? f(d, std::true_type{}) : f(d, std::false_type{}); };
  switch (D) {
    case 16: return go(std::integral_constant<int, 16>{});
    case 32: return go(std::integral_constant<int, 32>{});
    case 64: return go(std::integral_constant<int, 64>{});
    case 128: return go(std::integral_constant<int, 128>{});
  }
  return cudaErrorInvalidValue;
}

size_t table_bytes(const NormRopeParams& p) {
  return p.P == 0 ? 0 : static_cast<size_t>(p.tile) * 2 * (p.interleaved ? p.D / 2 : p.P) * sizeof(float);
}

}  // namespace

// Work split.  Warps: up to 8 groups a CTA; where there are fewer, `parts`
// warps share a group's tokens.  Tile: 8 rows a lane or more and 4 angles a
// thread, at most 16 KB of angles; halved while the tiles do not give every SM
// two CTAs.  The backward's CTAs stay for all of their tiles: one wave of
// them, and the tile size (of three) that leaves the least of it idle.
void norm_rope_plan(NormRopeParams* p, bool backward) {
  p->groups = groups_of(p->side[0].H, p->D) + groups_of(p->side[1].H, p->D);
  p->ctas_y = (p->groups + kMaxWarps - 1) / kMaxWarps;
  p->cta_groups = (p->groups + p->ctas_y - 1) / p->ctas_y;
  p->parts = kMaxWarps / p->cta_groups;
  const int warps = p->cta_groups * p->parts;
  int tt = 1;
  for (const NormRopeSide& s : p->side)
    if (s.H) tt = std::max(tt, 256 / p->D / heads_per_group(s.H, p->D));
  const long width = p->interleaved ? p->D / 2 : p->P;
  long t = 8L * tt * p->parts;
  while (t * width < 4 * 32 * warps && width > 0) t *= 2;
  while (t > 1 && t * width * 8 > 16384) t /= 2;
  auto tiles = [&](long tile) { return static_cast<long>(p->B) * ((p->N + tile - 1) / tile); };
  while (t > 1 && tiles(t) * p->ctas_y < 2 * kNumSM) t /= 2;
  if (backward) {
    const long slots = std::max(1L, static_cast<long>(kNumSM) * (kWarpsPerSM / warps) / p->ctas_y);
    long best = t, best_cost = -1;
    for (long c = t, k = 0; c >= 1 && k < 3; c /= 2, ++k) {
      const long cost = (tiles(c) + slots - 1) / slots * (c + tt * p->parts);
      if (best_cost < 0 || cost < best_cost) {
        best_cost = cost;
        best = c;
      }
    }
    t = best;
    p->ranges = static_cast<int>(std::min(slots, tiles(t)));
  }
  p->tile = static_cast<int>(t);
  p->tiles_per_b = static_cast<int>((p->N + t - 1) / t);
  p->n_tiles = tiles(t);
}

size_t norm_rope_part_floats(long B, long N, long Hq, long Hk, long D) {
  NormRopeParams p{};
  p.B = static_cast<int>(B);
  p.N = static_cast<int>(N);
  p.D = static_cast<int>(D);
  p.side[0].H = static_cast<int>(Hq);
  p.side[1].H = static_cast<int>(Hk);
  // a range has at least one token
  norm_rope_plan(&p, true);
  const long slots = std::max(1L, static_cast<long>(kNumSM) * (kWarpsPerSM / (p.cta_groups * p.parts)) / p.ctas_y);
  return static_cast<size_t>(std::min(slots, B * N)) * p.ctas_y * (Hq + Hk) * D;
}

cudaError_t launch_norm_rope_fwd(const NormRopeParams& p, cudaStream_t s) {
  return by_dim(p.D, p.interleaved, [&](auto d, auto il) {
    norm_rope_fwd_kernel<decltype(d)::value, decltype(il)::value>
        <<<static_cast<unsigned>(p.n_tiles * p.ctas_y), 32 * p.cta_groups * p.parts, table_bytes(p), s>>>(p);
    return cudaGetLastError();
  });
}

cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, cudaStream_t s) {
  const cudaError_t e = by_dim(p.D, p.interleaved, [&](auto d, auto il) {
    norm_rope_bwd_kernel<decltype(d)::value, decltype(il)::value>
        <<<static_cast<unsigned>(static_cast<long>(p.ranges) * p.ctas_y), 32 * p.cta_groups * p.parts, table_bytes(p), s>>>(p);
    return cudaGetLastError();
  });
  const int cols = gain_cols(p.side[0], p.D) + gain_cols(p.side[1], p.D);
  if (e != cudaSuccess || cols == 0) return e;
  gain_sum_kernel<<<(cols + 31) / 32, dim3(32, 32), 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace flare
