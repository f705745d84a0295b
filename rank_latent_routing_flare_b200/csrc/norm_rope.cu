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
// and one write).  A lane holds 16 elements, D / 16 lanes a row, in two
// 16-byte pieces chosen so that both members of a pair are the lane's own:
// the rotation needs no exchange, and the row's sums are a few shuffles.  The input
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
//
// Measured: keys of 8 heads of 16, 2^20 points in space, 121 us (4.5 TB/s); 32 x
// 4096 tokens, 8 + 8 heads of 32, padded, 52 us (4.2); backward of 32 + 8 heads
// of 128, 2 x 8191 tokens, 132 us (3.8), of 8 + 8 heads of 16, 4 x 65536 points, 96
// us (4.2).  The same accesses without arithmetic take 95, 47, 93 and 78 us: short
// rows and two strides keep them from the 6.5 TB/s of a plain copy.
#include <algorithm>

#include "flare_internal.h"
#include "norm_rope.h"
#include "ptx.cuh"

namespace flare {
namespace {

constexpr int kMaxWarps = 8;
constexpr int kWarpsPerSM = 16;   // resident at 128 registers a thread
constexpr int kTableBytes = 16384; // of one tile's angles, at most
constexpr int kRedCols = 128;     // columns of a group: ht * D
constexpr int kTablePad = 4;

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

// Walks a CTA's tiles: range, range + ranges, ...
struct Walk {
  long tile;
  int b, n0, ntok, nvalid;   // tokens n0 .. n0 + ntok of entry b, the first nvalid of them not padding
  __device__ __forceinline__ void open(const NormRopeParams& p) {
    ntok = nvalid = 0;
    if (tile >= p.n_tiles) return;
    b = static_cast<int>(tile / p.tiles_per_b);
    n0 = static_cast<int>(tile - static_cast<long>(b) * p.tiles_per_b) * p.tile;
    ntok = min(p.tile, p.N - n0);
    nvalid = p.lengths == nullptr ? ntok : max(0, min(ntok, p.lengths[b] - n0));
  }
};

// Positions of a tile's tokens into shared memory, asynchronously.
__device__ __forceinline__ void copy_positions(const NormRopeParams& p, const Walk& w, float* dst) {
  if (p.pos_kind != 0) {
    const float* src = static_cast<const float*>(p.pos) + (static_cast<long>(w.b) * p.N + w.n0) * p.axes;
    for (int i = threadIdx.x; i < w.nvalid * p.axes; i += blockDim.x)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst + i)), "l"(src + i) : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void wait_positions() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// cos and sin of the tile's first `nvalid` tokens: cs[token][cos W | sin W | pad].
// The padding puts the pieces that the tokens of a warp read on different banks.
template <int D, bool IL>
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, const Walk& w, const float* pos, float* cs) {
  const int W = table_width<D, IL>(p.P);
  const int bits = W <= 1 ? 0 : 32 - __clz(W - 1);          // a thread keeps one pair
  const int q = threadIdx.x & ((1 << bits) - 1), step = blockDim.x >> bits, t0 = threadIdx.x >> bits;
  if (q >= W || t0 >= step) return;
  double f[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    f[k] = k < p.axes && q < p.P ? static_cast<double>(p.freqs[k * p.P + q]) * 0.15915494309189533577 : 0.0;   // turns
  for (int t = t0; t < w.nvalid; t += step) {
    double a;
    if (p.pos_kind == 2) {
      a = static_cast<double>(pos[t * p.axes]) * f[0];
#pragma unroll
      for (int k = 1; k < 4; ++k)
        if (k < p.axes) a = fma(static_cast<double>(pos[t * p.axes + k]), f[k], a);
    } else {
      a = static_cast<double>(p.pos_kind == 1 ? __float_as_int(pos[t]) : w.n0 + t) * f[0];
    }
    a -= rint(a);
    float sn, cn;
    sincospif(2.0f * static_cast<float>(a), &sn, &cn);
    cs[t * (2 * W + kTablePad) + q] = cn;
    cs[t * (2 * W + kTablePad) + W + q] = sn;
  }
}

// 16 elements of a row: two pieces of 8, each as four fp32 pairs.
struct Vec16 {
  uint64_t v[8];
};
__device__ __forceinline__ void unpack8(const uint4& r, uint64_t* v) {
  v[0] = f2_pack(bf16_lo(r.x), bf16_hi(r.x));
  v[1] = f2_pack(bf16_lo(r.y), bf16_hi(r.y));
  v[2] = f2_pack(bf16_lo(r.z), bf16_hi(r.z));
  v[3] = f2_pack(bf16_lo(r.w), bf16_hi(r.w));
}
__device__ __forceinline__ uint32_t round_pair(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint4 pack8(const uint64_t* v) {
  return make_uint4(round_pair(v[0]), round_pair(v[1]), round_pair(v[2]), round_pair(v[3]));
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_dup(float a) { return f2_pack(a, a); }
__device__ __forceinline__ void load_gain8(const float* g, uint64_t* v) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(g)), b = __ldg(reinterpret_cast<const float4*>(g) + 1);
  v[0] = f2_pack(a.x, a.y);
  v[1] = f2_pack(a.z, a.w);
  v[2] = f2_pack(b.x, b.y);
  v[3] = f2_pack(b.z, b.w);
}
__device__ __forceinline__ float dot16(const Vec16& a, const Vec16& b) {
  uint64_t s = f2_mul(a.v[0], b.v[0]), u = f2_mul(a.v[4], b.v[4]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    s = f2_fma(a.v[i], b.v[i], s);
    u = f2_fma(a.v[4 + i], b.v[4 + i], u);
  }
  float lo, hi;
  f2_unpack(f2_add(s, u), lo, hi);
  return lo + hi;
}
template <int D>
__device__ __forceinline__ float row_sum(float v) {   // over the D / 16 lanes of a row
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// A lane's place in its warp's group of rows: token t_in of tt, head h_in of
// ht, and two pieces of 8 elements from e0 and e1: half-split pairs have one
// member in each (pairs first .. first + 7), interleaved pairs lie within the
// 16 consecutive elements (pairs first .. first + 7 too).
template <int D, bool IL>
struct Place {
  int ht, tt, h_in, t_in, e0, e1, first;
  bool turned;
  __device__ __forceinline__ Place(int H, int lane, int P) {
    constexpr int L = D / 16;
    ht = heads_per_group(H, D);
    tt = (32 / L) / ht;
    const int l = lane % L, rr = lane / L;
    h_in = rr & (ht - 1);
    t_in = rr / ht;
    if (IL) {
      e0 = 16 * l;
      e1 = e0 + 8;
      first = 8 * l;
      turned = first < P;
    } else {
      const int ph = P / 8;
      turned = l < ph;
      e0 = turned ? 8 * l : 16 * l;   // lanes behind the pairs' take the rest, 16 elements each: 2 P + 16 (l - ph)
      e1 = turned ? P + 8 * l : e0 + 8;
      first = 8 * l;
    }
  }
};
// The pairs of a lane turned by the angles of a token (dir 1) or back (-1).
template <bool IL>
__device__ __forceinline__ void rotate(Vec16& x, const float* cs, int W, float dir) {
  const float4* c4 = reinterpret_cast<const float4*>(cs);
  const float4* s4 = reinterpret_cast<const float4*>(cs + W);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 c = c4[i], s = s4[i];
    if (IL) {
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint64_t& v = x.v[4 * i + k];
        float a, b;
        f2_unpack(v, a, b);
        v = f2_fma(f2_pack(b, a), f2_pack(-dir * ss[k], dir * ss[k]), f2_mul(v, f2_dup(cc[k])));
      }
    } else {
      const uint64_t cc[2] = {f2_pack(c.x, c.y), f2_pack(c.z, c.w)};
      const uint64_t ss[2] = {f2_pack(dir * s.x, dir * s.y), f2_pack(dir * s.z, dir * s.w)};
      const uint64_t ns[2] = {f2_pack(-dir * s.x, -dir * s.y), f2_pack(-dir * s.z, -dir * s.w)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint64_t& a = x.v[2 * i + k];
        uint64_t& b = x.v[4 + 2 * i + k];
        const uint64_t ta = f2_fma(b, ns[k], f2_mul(a, cc[k]));
        b = f2_fma(a, ss[k], f2_mul(b, cc[k]));
        a = ta;
      }
    }
  }
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

// Columns of a side's gain gradient in a CTA's partial row.
__host__ __device__ inline int gain_cols(const NormRopeSide& s, int D) {
  return s.dgain ? (s.gain_per_head ? s.H * D : D) : 0;
}

// A CTA's partial row of the gains' gradients: the lanes of one head, then the
// warps, in a fixed order.
template <int D, bool IL>
__device__ __forceinline__ void gain_row(const NormRopeParams& p, float (*red)[kRedCols], const Place<D, IL>& at, const Vec16& dg) {
  const int warp = threadIdx.x >> 5;
  const int cq = gain_cols(p.side[0], D), cols = cq + gain_cols(p.side[1], D);
  if (cols == 0) return;
  __syncthreads();   // red lies over the tables
  float f[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) f2_unpack(dg.v[i], f[2 * i], f[2 * i + 1]);
  for (int o = at.ht * (D / 16); o < 32; o <<= 1) {
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] += __shfl_xor_sync(~0u, f[e], o);
  }
  if (at.t_in == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      red[warp][at.h_in * D + at.e0 + e] = f[e];
      red[warp][at.h_in * D + at.e1 + e] = f[8 + e];
    }
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

// Both directions.  Positions come to shared memory two tiles ahead; a tile's
// first rows are requested before its angles are computed.  Two angle tables and two position buffers:
// one barrier a tile.
template <int D, bool IL, bool BWD>
__global__ void __launch_bounds__(32 * kMaxWarps, kWarpsPerSM / kMaxWarps) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  extern __shared__ __align__(16) float smem[];
  constexpr int U = BWD ? 1 : 2;   // rows a lane requests at once
  const int lane = threadIdx.x & 31;
  const int range = static_cast<int>(blockIdx.x / p.ctas_y);
  const Unit unit = warp_unit(p);
  const bool active = unit.side >= 0;
  const NormRopeSide& s = p.side[max(unit.side, 0)];
  const Place<D, IL> at(max(s.H, 1), lane, p.P);
  const int W = table_width<D, IL>(p.P), row = 2 * W + kTablePad, table = p.tile * row;
  const int head = unit.group * at.ht + at.h_in;
  const int step = p.parts * at.tt, t_first = unit.part * at.tt + at.t_in;
  const uint16_t* x0 = s.x + head * s.xs[1] + at.e0;
  const uint16_t* d0 = BWD ? s.dy + head * s.ds[1] + at.e0 : nullptr;
  uint16_t* y0 = s.y + head * s.ys[1] + at.e0;
  const int other = at.e1 - at.e0;

  Vec16 g, dg;
  const float* gp = s.gain + (s.gain_per_head ? static_cast<long>(head) * D : 0);
  if (s.gain) {
    load_gain8(gp + at.e0, g.v);
    load_gain8(gp + at.e1, g.v + 4);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!s.gain) g.v[i] = f2_dup(1.f);
    dg.v[i] = f2_dup(0.f);
  }

  float* pos = smem + 2 * table;
  const int pos_floats = p.tile * p.axes;
  uint4 rx[U][2], rd[U][2];
  Walk w, next;
  const uint16_t *x, *d;
  auto fetch = [&](const Walk& at_tile, int t0) {   // a lane's next U rows
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * step;
#pragma unroll
      for (int i = 0; i < 2; ++i) rx[u][i] = rd[u][i] = make_uint4(0, 0, 0, 0);
      if (active && t < at_tile.nvalid) {
        rx[u][0] = *reinterpret_cast<const uint4*>(x + t * s.xs[2]);
        rx[u][1] = *reinterpret_cast<const uint4*>(x + t * s.xs[2] + other);
        if (BWD) {
          rd[u][0] = *reinterpret_cast<const uint4*>(d + t * s.ds[2]);
          rd[u][1] = *reinterpret_cast<const uint4*>(d + t * s.ds[2] + other);
        }
      }
    }
  };
  auto begin = [&](const Walk& at_tile) {           // a tile's first rows
    if (at_tile.ntok == 0) return;
    x = x0 + at_tile.b * s.xs[0] + static_cast<long>(at_tile.n0) * s.xs[2];
    if (BWD) d = d0 + at_tile.b * s.ds[0] + static_cast<long>(at_tile.n0) * s.ds[2];
    fetch(at_tile, t_first);
  };
  auto copy = [&](int k, Walk at_tile) {            // positions of the CTA's k-th tile
    copy_positions(p, at_tile, pos + (k & 1) * pos_floats);
  };
  auto after = [&](Walk at_tile) {
    at_tile.tile += p.ranges;
    at_tile.open(p);
    return at_tile;
  };
  next.tile = range;
  next.open(p);
  begin(next);
  if (p.P > 0) {
    copy(0, next);
    copy(1, after(next));
    wait_positions();
    __syncthreads();
    fill_angles<D, IL>(p, next, pos, smem);
  }
  for (int k = 0; next.ntok > 0; ++k) {
    w = next;
    next = after(w);
    const float* cs = smem + (k & 1) * table;
    if (p.P > 0) {
      // behind the barrier: this tile's angles, the next tile's positions, and
      // every warp done with the tile before
      wait_positions();
      __syncthreads();
      copy(k, after(next));   // k + 2
    }
    uint16_t* y = y0 + w.b * s.ys[0] + static_cast<long>(w.n0) * s.ys[2];
    for (int t0 = t_first; active && t0 - at.t_in < w.ntok; t0 += U * step) {
      Vec16 v[U], u[BWD ? U : 1];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        unpack8(rx[i][0], v[i].v);
        unpack8(rx[i][1], v[i].v + 4);
        if constexpr (BWD) {
          unpack8(rd[i][0], u[i].v);
          unpack8(rd[i][1], u[i].v + 4);
        }
      }
      if (t0 + U * step - at.t_in < w.ntok) fetch(w, t0 + U * step); else begin(next);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int t = t0 + i * step;
        if (t - at.t_in >= w.ntok) break;   // uniform over the warp
        Vec16& x16 = v[i];
        // 0 for a lane without a row: it adds nothing to the gains' gradients, whatever eps is
        const float mean = fmaf(row_sum<D>(dot16(x16, x16)), 1.0f / D, p.eps), r = t < w.nvalid ? rsqrtf(mean) : 0.f;
        const uint64_t r2 = f2_dup(r);
        if constexpr (!BWD) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x16.v[e] = f2_mul(f2_mul(x16.v[e], r2), g.v[e]);
          if (at.turned && t < w.nvalid) rotate<IL>(x16, cs + t * row + at.first, W, 1.f);
        } else {
          Vec16& u16 = u[i];
          if (at.turned && t < w.nvalid) rotate<IL>(u16, cs + t * row + at.first, W, -1.f);
          uint64_t sum2 = f2_dup(0.f);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum2 = f2_fma(f2_mul(u16.v[e], g.v[e]), x16.v[e], sum2);   // <w, x>
          float s0, s1;
          f2_unpack(sum2, s0, s1);
          const uint64_t k2 = f2_dup(-r * r * row_sum<D>(s0 + s1) * (1.0f / D));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dg.v[e] = f2_fma(u16.v[e], f2_mul(x16.v[e], r2), dg.v[e]);
            x16.v[e] = f2_mul(r2, f2_fma(x16.v[e], k2, f2_mul(u16.v[e], g.v[e])));
          }
        }
        if (t < w.ntok) {
          const bool live = t < w.nvalid;
          uint16_t* dst = y + t * s.ys[2];
          *reinterpret_cast<uint4*>(dst) = live ? pack8(x16.v) : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(dst + other) = live ? pack8(x16.v + 4) : make_uint4(0, 0, 0, 0);
        }
      }
    }
    if (t_first - at.t_in >= w.ntok) begin(next);   // a share without tokens in a short tile
    if (p.P > 0) fill_angles<D, IL>(p, next, pos + ((k + 1) & 1) * pos_floats, smem + ((k + 1) & 1) * table);
  }
  if constexpr (BWD) gain_row<D, IL>(p, reinterpret_cast<float(*)[kRedCols]>(smem), at, dg);
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

// CTAs over the tiles in one wave.
long range_slots(const NormRopeParams& p) {
  return std::max(1L, static_cast<long>(kNumSM) * (kWarpsPerSM / (p.cta_groups * p.parts)) / p.ctas_y);
}

// Two tables of angles and two buffers of positions; in the backward the warps' gradient sums lie over them.
size_t smem_bytes(const NormRopeParams& p, bool backward) {
  const size_t row = 2 * (p.interleaved ? p.D / 2 : p.P) + kTablePad;
  const size_t tables = p.P == 0 ? 0 : 2 * static_cast<size_t>(p.tile) * (row + p.axes) * sizeof(float);
  return std::max(tables, backward ? kMaxWarps * kRedCols * sizeof(float) : 0);
}

template <bool BWD>
cudaError_t launch(const NormRopeParams& p, cudaStream_t s) {
  const size_t smem = smem_bytes(p, BWD);   // at most 2 (kTableBytes + 8 floats a token)
  return by_dim(p.D, p.interleaved, [&](auto d, auto il) {
    norm_rope_kernel<decltype(d)::value, decltype(il)::value, BWD>
        <<<static_cast<unsigned>(static_cast<long>(p.ranges) * p.ctas_y), 32 * p.cta_groups * p.parts, smem, s>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace

// Work split.  Warps: up to 8 groups a CTA; where there are fewer, `parts`
// warps share a group's tokens.  One wave of CTAs, each with every ranges-th
// tile.  Tile: 8 rows a lane or more, 4 angles a thread and kTableBytes of
// angles at most; halved while the tiles do not give every SM two CTAs, and
// then the size (of three) that leaves the least of the wave idle.
void norm_rope_plan(NormRopeParams* p) {
  p->groups = groups_of(p->side[0].H, p->D) + groups_of(p->side[1].H, p->D);
  p->ctas_y = (p->groups + kMaxWarps - 1) / kMaxWarps;
  p->cta_groups = (p->groups + p->ctas_y - 1) / p->ctas_y;
  p->parts = kMaxWarps / p->cta_groups;
  const int warps = p->cta_groups * p->parts;
  int tt = 1;
  for (const NormRopeSide& s : p->side)
    if (s.H) tt = std::max(tt, 512 / p->D / heads_per_group(s.H, p->D));
  const long width = p->interleaved ? p->D / 2 : p->P;
  long t = 8L * tt * p->parts;
  while (t * width < 4 * 32 * warps && width > 0) t *= 2;
  while (t > 1 && t * width * 8 > kTableBytes) t /= 2;
  auto tiles = [&](long tile) { return static_cast<long>(p->B) * ((p->N + tile - 1) / tile); };
  while (t > 1 && tiles(t) * p->ctas_y < 2 * kNumSM) t /= 2;
  const long slots = range_slots(*p);
  long best = t, best_cost = -1;
  for (long c = t, k = 0; c >= 1 && k < 3; c /= 2, ++k) {
    const long cost = (tiles(c) + slots - 1) / slots * (c + tt * p->parts);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = c;
    }
  }
  p->tile = static_cast<int>(best);
  p->tiles_per_b = static_cast<int>((p->N + best - 1) / best);
  p->n_tiles = tiles(best);
  p->ranges = static_cast<int>(std::min(slots, p->n_tiles));
}

size_t norm_rope_part_floats(long B, long N, long Hq, long Hk, long D) {
  NormRopeParams p{};
  p.B = static_cast<int>(B);
  p.N = static_cast<int>(N);
  p.D = static_cast<int>(D);
  p.side[0].H = static_cast<int>(Hq);
  p.side[1].H = static_cast<int>(Hk);
  norm_rope_plan(&p);
  return static_cast<size_t>(std::min(range_slots(p), B * N)) * p.ctas_y * (Hq + Hk) * D;   // a tile has a token at least
}

cudaError_t launch_norm_rope_fwd(const NormRopeParams& p, cudaStream_t s) { return launch<false>(p, s); }

cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, cudaStream_t s) {
  const cudaError_t e = launch<true>(p, s);
  const int cols = gain_cols(p.side[0], p.D) + gain_cols(p.side[1], p.D);
  if (e != cudaSuccess || cols == 0) return e;
  gain_sum_kernel<<<(cols + 31) / 32, dim3(32, 32), 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace flare
