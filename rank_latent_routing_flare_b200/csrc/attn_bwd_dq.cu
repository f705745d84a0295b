// The dQ pass of the attention's backward, and the row statistics both passes
// read.
#include "attn_bwd_kernel.cuh"

namespace flare {
namespace {

// A row's largest score, in log2 units over biased positions, by the row's
// lanes, a key each.  It stands in for the log-sum-exp of a row so far from
// its keys that L, about -slope times that distance, has no bits left for the
// scores (the dQ pass divides by the sum of the weights in any case).  Slow,
// and rare: a row 2^24 / slope tokens or more from the nearest key it sees.
constexpr float kFarBias = 0x1p24f;   // up to here L is off by a few units, weights by e^3
template <int D>
__device__ __noinline__ float largest_score(const AttnBwdParams& bp, int b, int h, int i, int2 iv, int pos, int l) {
  const AttnParams& p = bp.a;
  const ScoreOps ops(p.scale, p.cap, true);
  const uint4* q = reinterpret_cast<const uint4*>(bp.q.p + b * bp.q.sb + h * bp.q.sh + i * bp.q.sn);
  const uint16_t* k = bp.k.p + b * bp.k.sb + h / p.G * bp.k.sh;
  float top = -INFINITY;
  for (int j = iv.x + l; j < iv.y; j += D / 8) {
    const uint4* kj = reinterpret_cast<const uint4*>(k + j * bp.k.sn);
    float s = 0.f;
#pragma unroll 2
    for (int c = 0; c < D / 8; ++c) {
      const uint4 x = q[c], y = kj[c];
      const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) s = fmaf(bf16_lo(u[e]), bf16_lo(v[e]), fmaf(bf16_hi(u[e]), bf16_hi(v[e]), s));
    }
    s = p.cap > 0.f ? ops.capped(s) : s * ops.c2;
    top = fmaxf(top, fmaf(-p.slopes[h] * kLog2e, fabsf(static_cast<float>(pos - j)), s));
  }
  return top;
}

// One row's statistics: l2 = L log2(e), moved by the distance that the bias
// positions leave out, and delta = <dY, Y> in fp32.  D / 8 lanes a row, 16-byte
// loads.
template <int D, bool BIAS>
__global__ void __launch_bounds__(256) attn_rows_kernel(const __grid_constant__ AttnBwdParams bp) {
  constexpr int L = D / 8, ROWS = 256 / L, T = BwdCfg<D, true>::T;
  const AttnParams& p = bp.a;
  const int rows = bp.row_blocks * T, blocks = (rows + ROWS - 1) / ROWS;
  const long bh = blockIdx.x / blocks;
  const int i = static_cast<int>(blockIdx.x - bh * blocks) * ROWS + threadIdx.x / L, l = threadIdx.x % L;
  const int b = static_cast<int>(bh / p.Hq), h = static_cast<int>(bh % p.Hq);
  if (blockIdx.x == 0 && threadIdx.x < 4) p.err[threadIdx.x] = 0u;
  const BatchMask m = batch_mask(p.mask, b);
  const int2 iv = row_interval(m, i);
  const bool sees = i < p.mask.Nq && iv.x < iv.y;
  float delta = 0.f;
  if (sees) {
    const uint4 a = *reinterpret_cast<const uint4*>(bp.dy.p + b * bp.dy.sb + h * bp.dy.sh + i * bp.dy.sn + 8 * l);
    const uint4 y = *reinterpret_cast<const uint4*>(bp.yin.p + b * bp.yin.sb + h * bp.yin.sh + i * bp.yin.sn + 8 * l);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) delta = fmaf(bf16_lo(u[k]), bf16_lo(v[k]), fmaf(bf16_hi(u[k]), bf16_hi(v[k]), delta));
  }
  const int pos = bias_position(m, i, iv);
  bool far = false;
  float top = 0.f;
  if constexpr (BIAS) {
    far = sees && fabsf(p.slopes[h] * bias_shift(m, i, iv)) > kFarBias;
    if (far) top = largest_score<D>(bp, b, h, i, iv, pos, l);
    __syncwarp();
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) delta += __shfl_xor_sync(~0u, delta, o);
  if (l == 0 && i < rows) {
    float l2 = INFINITY;
    if (sees) {
      float L2 = p.L[bh * p.mask.Nq + i];
      if (BIAS) L2 += p.slopes[h] * bias_shift(m, i, iv);
      if (far) l2 = top;
      else if (L2 != -INFINITY) l2 = L2 * kLog2e;
    }
    float* r = bp.rows + (bh * bp.row_blocks + i / T) * (kAttnRowFields * T) + i % T;
    r[0] = -l2;
    r[T] = l2 == INFINITY ? 0.f : -delta;
    r[2 * T] = __int_as_float(iv.x);
    r[3 * T] = __int_as_float(iv.y);
    r[4 * T] = __int_as_float(pos);
  }
}

}  // namespace

int attn_bwd_stream_tile(int D, bool kv) {
  return D == 128  ? (kv ? BwdCfg<128, true>::T : BwdCfg<128, false>::T)
         : D == 64 ? (kv ? BwdCfg<64, true>::T : BwdCfg<64, false>::T)
                   : (kv ? BwdCfg<32, true>::T : BwdCfg<32, false>::T);
}

bool attn_bwd_rows_in_tmem(int D, bool kv) {
  return D == 128 ? (kv ? BwdCfg<128, true>::XT : BwdCfg<128, false>::XT) : D == 64 && (kv ? BwdCfg<64, true>::XT : BwdCfg<64, false>::XT);
}

cudaError_t launch_attn_rows(const AttnBwdParams& p, cudaStream_t s) {
  auto go = [&](auto d) {
    constexpr int D = decltype(d)::value, ROWS = 256 / (D / 8);
    const long blocks = (static_cast<long>(p.row_blocks) * BwdCfg<D, true>::T + ROWS - 1) / ROWS;
    const unsigned grid = static_cast<unsigned>(blocks * p.a.B * p.a.Hq);
    if (p.a.slopes) attn_rows_kernel<D, true><<<grid, 256, 0, s>>>(p);
    else attn_rows_kernel<D, false><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
  };
  switch (p.a.D) {
    case 16: return go(std::integral_constant<int, 16>{});
    case 32: return go(std::integral_constant<int, 32>{});
    case 64: return go(std::integral_constant<int, 64>{});
    case 128: return go(std::integral_constant<int, 128>{});
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_attn_bwd_dq(const AttnMaps& m, const AttnBwdParams& p, cudaStream_t s) {
  return launch_attn_bwd_pass<false>(m.q, m.dy, m.k, m.v, p, s);
}

}  // namespace flare
