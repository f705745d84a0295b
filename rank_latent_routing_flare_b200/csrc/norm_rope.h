// Parameters of the query/key preparation kernels (norm_rope.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace flare {

// One of the two tensors: queries or keys (H = 0: absent).
struct NormRopeSide {
  int H;
  int gain_per_head;
  const uint16_t* x;    // input rows
  const uint16_t* dy;   // backward: gradient of the output rows
  uint16_t* y;          // forward: output rows; backward: dx
  const float* gain;    // [D] or [H][D], or nullptr
  float* dgain;         // backward: gradient of the gain, or nullptr
  long xs[3], ds[3], ys[3];  // strides in elements: batch, head, row
};

struct NormRopeParams {
  NormRopeSide side[2];
  int B, N, D;
  int P;                // rotated pairs
  int axes, pos_kind, interleaved;
  const float* freqs;   // [axes][P]
  const void* pos;
  const int32_t* lengths;
  float eps;
  int tile;             // tokens per tile
  int tiles_per_b;
  long n_tiles;         // B * tiles_per_b
  int ctas;             // backward: CTAs launched
  float* part;          // backward: [ctas][(Hq + Hk) D] partial sums of the gains' gradients
};

// Upper bound of the backward's CTAs for these sizes (sizes its workspace).
int norm_rope_bwd_ctas(long B, long N);
// Chooses tile, tiles_per_b, n_tiles and ctas.
void norm_rope_plan(NormRopeParams* p, bool backward);
cudaError_t launch_norm_rope_fwd(const NormRopeParams& p, cudaStream_t s);
cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, cudaStream_t s);

}  // namespace flare
