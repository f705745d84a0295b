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
  // work split (norm_rope_plan)
  int groups;           // groups of heads a warp takes at once, queries' first
  int ctas_y;           // CTAs over the groups
  int cta_groups;       // groups per CTA
  int parts;            // shares of a tile's tokens per group: warps per CTA = cta_groups * parts
  int tile;             // tokens per tile
  int tiles_per_b;
  long n_tiles;         // B * tiles_per_b
  int ranges;           // CTAs over the tiles, each taking every ranges-th
  float* part;          // backward: [ranges][ctas_y][gain columns] partial sums of the gains' gradients
};

// Floats of partial sums the backward may need for these sizes.
size_t norm_rope_part_floats(long B, long N, long Hq, long Hk, long D);
// Chooses the work split.
void norm_rope_plan(NormRopeParams* p);
cudaError_t launch_norm_rope_fwd(const NormRopeParams& p, cudaStream_t s);
cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, cudaStream_t s);

}  // namespace flare
