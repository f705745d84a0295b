// Parameters of the exact softmax attention kernels (attn_fwd.cu,
// attn_step.cu, attn_bwd_dq.cu, attn_bwd_dkv.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace flare {

// Masks.  Every mask leaves row i of a batch entry one interval [lo, hi) of
// keys, and lo and hi do not decrease with i: the rows that see a key tile
// and the keys that a row tile sees are ranges too.
struct AttnMask {
  int Nq, Nk, causal;
  const int32_t *lengths, *q_lengths, *q_offsets, *prefix;
  const int2* doc;   // [B][Nk] first and one-past-last position of the document a position lies in
                     // (equal: in none), or nullptr
};

struct AttnSide {    // rows [B][H][N][D] with strides in elements
  const uint16_t* p;
  long sb, sh, sn;
};

constexpr int kAttnClusterSplits = 8;   // portable cluster size

struct AttnParams {
  int B, Hq, Hk, G, D;           // G = Hq / Hk
  AttnMask mask;
  float scale;                   // applied to <q, k>
  float cap;                     // <= 0: none
  const float* slopes;           // [Hq] or nullptr
  uint16_t* y;
  long ys[3];
  float* L;                      // [B][Hq][Nq] or nullptr
  // work split along the keys: up to kAttnClusterSplits splits are a cluster
  // that joins in shared memory; more leave partial results for attn_join
  int splits;
  float* part_o;                 // [splits][B][Hq][Nq][D], each split's normalised output
  float* part_l;                 // [splits][B][Hq][Nq], its log2 sum of weights
  uint32_t* err;
  unsigned long long timeout_ns;
};

// Statistics of the backward's query rows: per batch entry and query head,
// blocks of T = attn_bwd_stream_tile(D, true) rows, each kAttnRowFields arrays of T
// 4-byte values: -l2 (P = 2^(x - l2); -inf: the row sees nothing), -delta
// (delta = <dY, Y>), the interval [lo, hi) of keys that it sees, and its
// position for the distance bias.
constexpr int kAttnRowFields = 5;

struct AttnBwdParams {
  AttnParams a;
  AttnSide q, k, v, dy, yin;
  uint16_t *dq, *dk, *dv;
  long dqs[3], dks[3], dvs[3];
  float* rows;
  int row_blocks;                // blocks per head
  int split_bits;                // dK/dV pass: log2 of the CTAs that share a key tile's stream
};

struct AttnMaps {                // tensor maps of the kernels' operands
  CUtensorMap q, k, v, dy;
};

// Runs of equal ids -> the document table of AttnMask.
cudaError_t launch_attn_documents(const int32_t* ids, int2* doc, int B, int N, cudaStream_t s);

int attn_fwd_key_tile(int D, bool bias, bool cap);   // keys per tile; the query tile is kAttnQTile rows
constexpr int kAttnQTile = 128;
cudaError_t launch_attn_fwd(const AttnMaps& m, const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_join(const AttnParams& p, cudaStream_t s);

constexpr int kAttnStepRows = 16;   // query rows per key head of the kernel for few rows
cudaError_t launch_attn_step(const AttnParams& p, const AttnSide& q, const AttnSide& k, const AttnSide& v,
                             cudaStream_t s);

int attn_step_ctas(int D);                  // CTAs of the few-row kernel that share an SM
int attn_bwd_stream_tile(int D, bool kv);   // rows per streamed tile of the dQ pass and of the dK/dV pass
bool attn_bwd_rows_in_tmem(int D, bool kv);  // whether a pass reads its own tile of rows without a map
cudaError_t launch_attn_rows(const AttnBwdParams& p, cudaStream_t s);
cudaError_t launch_attn_bwd_dq(const AttnMaps& m, const AttnBwdParams& p, cudaStream_t s);
cudaError_t launch_attn_bwd_dkv(const AttnMaps& m, const AttnBwdParams& p, cudaStream_t s);

}  // namespace flare
