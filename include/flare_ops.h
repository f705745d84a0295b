/*
 * flare_ops.h - C ABI of the operators around the FLARE / FLARE++ mixer on
 * B200 (sm_100a): the preparation of queries and keys (per-head RMS norm and
 * position rotation) and exact softmax attention, forward and backward.
 *
 * Conventions (status codes, flare_bf16, streams and workspaces as in
 * flare.h):
 *   - Tensors of rows are [B][H][N][D] bf16 in DEVICE memory with D dense
 *     elements per row and free strides over batch, head and row, given in
 *     elements: a head-major tensor has strides (H N D, N D, D), a slice of a
 *     token-major projection [B][N][Ht D] has (N Ht D, D, Ht D).  Every row
 *     starts on a 16-byte boundary (pointers aligned, strides multiples of 8
 *     elements, at most 2^38).  The stride of a size-one dimension is not read.
 *     A zero stride (an expanded tensor) is taken for inputs of the
 *     preparation and for Y, and refused elsewhere.  Outputs must not overlap
 *     each other or the inputs.
 *   - D in {16, 32, 64, 128}.
 *   - Arguments come in one struct whose members are all 8 bytes wide.
 *     Pointers marked optional may be NULL.
 *   - Every call only enqueues work on the stream (which must belong to the
 *     calling thread's current device) and may be captured into a graph;
 *     nothing is allocated and no state is kept between calls.  Two calls
 *     that may run at the same time need two workspaces.
 *   - Results are deterministic: no floating-point atomics.
 */
#ifndef FLARE_OPS_H_
#define FLARE_OPS_H_

#include "flare.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Preparation of queries and keys.  Per row x (one token n, one head h) of
 * Q and of K:
 *   y_d = x_d * rsqrt(mean_d(x^2) + eps) * gain_d
 *   then every pair (a, b) of y, p = 0 .. rot/2 - 1, is rotated:
 *   (a cos t - b sin t, a sin t + b cos t),  t = sum_i pos[n][i] * freqs[i][p]
 * The pairs are elements (p, p + rot/2), or (2p, 2p + 1) when interleaved;
 * elements rot .. D-1 are not rotated.  Angles are formed in 64 bits.
 *
 * Q or K may be absent (NULL with its outputs and gain NULL and its head
 * count 0).  rot = 0 (freqs NULL): norm only.  rot is even, at most D; a
 * multiple of 16 unless interleaved.
 *   pos_kind 0: pos[n] = n                          (axes 1, positions NULL)
 *   pos_kind 1: positions int32 [B][N]              (axes 1)
 *   pos_kind 2: positions float [B][N][axes]        (axes 1 .. 4)
 * gain: float [D], or [H][D] when gain_per_head; NULL: no gain.  Gains and
 * their gradients lie on 16-byte boundaries.
 * lengths: optional int32 [B], clamped to [0, N]; rows n >= lengths[b] are
 * not read and are written as zeros.
 */
typedef struct {
  int64_t B, N, D, Hq, Hk;
  int64_t rot, axes, interleaved, pos_kind;
  double eps;
  const float* freqs;      /* [axes][rot / 2] */
  const void* positions;
  const int32_t* lengths;
  const flare_bf16* Q;
  int64_t q_stride[3];     /* batch, head, row */
  const flare_bf16* K;
  int64_t k_stride[3];
  const float* q_gain;
  const float* k_gain;
  int64_t q_gain_per_head, k_gain_per_head;
  /* forward: Qr, Kr written; backward: their gradients, read */
  flare_bf16* Qr;
  int64_t qr_stride[3];
  flare_bf16* Kr;
  int64_t kr_stride[3];
  /* backward only: gradients, written; dq_gain, dk_gain are float tensors of the gains' shapes (NULL: not wanted) */
  flare_bf16* dQ;
  int64_t dq_stride[3];
  flare_bf16* dK;
  int64_t dk_stride[3];
  float* dq_gain;
  float* dk_gain;
} flare_qk_norm_rope_args;

/* Workspace of flare_qk_norm_rope_bwd (partial sums of the gains' gradients); 0 for unsupported sizes. */
FLARE_API size_t flare_qk_norm_rope_workspace_bytes(int64_t B, int64_t N, int64_t Hq, int64_t Hk, int64_t D);
FLARE_API flare_status flare_qk_norm_rope_fwd(const flare_qk_norm_rope_args* args, void* stream);
/*
 * Gradients: with g the gradient of a rotated row, u = g rotated back, r =
 * rsqrt(mean(x^2) + eps), w = u * gain:
 *   dx = r * (w - x r mean(w x r)),   dgain = sum over rows of u * x r
 * The workspace may be NULL when neither dq_gain nor dk_gain is wanted.
 */
FLARE_API flare_status flare_qk_norm_rope_bwd(const flare_qk_norm_rope_args* args, void* workspace,
                                              size_t workspace_bytes, void* stream);

/*
 * Exact softmax attention.  Query head h reads key head h / (Hq / Hk).  Row
 * i of Q stands at position p_i = q_offset + i.  Score of row i and key j:
 *   s = scale * <q_i, k_j>;  with cap > 0: s = cap * tanh(s / cap)
 *   with slopes: s -= slopes[h] * |p_i - j|
 * Row i sees key j when all of these hold:
 *   j < lengths[b], i < q_lengths[b]             (where given; clamped to [0, Nk] and [0, Nq])
 *   not causal, or j <= p_i, or j < prefix[b]
 *   no documents, or j and p_i lie in the same document: a document is a run
 *     of equal ids in documents[b][0 .. Nk); ids below zero belong to none
 * Y_i = softmax_j(s) V, L_i = log sum_j exp(s).  A row that sees no key has
 * Y_i = 0, L_i = -inf and zero gradients, and contributes none.
 *
 * Keys that no row sees (j >= lengths[b], ids below zero, other documents than
 * the rows', slots of a cache behind the newest token of a causal call) and
 * rows i >= q_lengths[b] may hold anything, infinities and NaN included.  A NaN
 * or an infinity in a row that takes part may also reach rows and keys that the
 * masks keep from it (0 times it is NaN, as in softmax(s) V).
 *
 * The scale is 0 or lies in [1e-30, 1e30], the cap is 0 or in [1e-6, 1e9]; Nq
 * and Nk are at most 2^27.  Products of bf16 rows, exponentials, sums and
 * statistics are fp32; weights and dS enter their products in bf16.  Gradients
 * with respect to the slopes are not computed.
 *
 * Workspaces hold an error word in front (flare_last_device_status), the
 * documents' intervals, the partial results of splits along the keys, or the
 * backward's row statistics.  Contents are not kept from call to call.
 */
typedef struct {
  int64_t B, Hq, Hk, Nq, Nk, D;
  int64_t causal;
  double scale;                /* <= 0: 1 / sqrt(D) */
  double cap;                  /* <= 0: not capped */
  const flare_bf16* Q;
  int64_t q_stride[3];
  const flare_bf16* K;
  int64_t k_stride[3];
  const flare_bf16* V;
  int64_t v_stride[3];
  const int32_t* lengths;      /* optional [B] */
  const int32_t* q_lengths;    /* optional [B] */
  const int32_t* q_offsets;    /* optional [B]; NULL: Nk - Nq */
  const int32_t* documents;    /* optional [B][Nk] */
  const int32_t* prefix;       /* optional [B]; read when causal */
  const float* slopes;         /* optional [Hq] */
  /* forward: written (L optional); backward: read */
  flare_bf16* Y;
  int64_t y_stride[3];
  float* L;                    /* [B][Hq][Nq] */
  /* backward only */
  const flare_bf16* dY;
  int64_t dy_stride[3];
  flare_bf16* dQ;
  int64_t dq_stride[3];
  flare_bf16* dK;
  int64_t dk_stride[3];
  flare_bf16* dV;
  int64_t dv_stride[3];
} flare_attention_args;

/* Workspace of flare_attention_fwd (backward = 0) or flare_attention_bwd (1); 0 for unsupported sizes. */
FLARE_API size_t flare_attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Hk, int64_t Nq, int64_t Nk, int64_t D,
                                                 int backward);
FLARE_API flare_status flare_attention_fwd(const flare_attention_args* args, void* workspace, size_t workspace_bytes,
                                           void* stream);
FLARE_API flare_status flare_attention_bwd(const flare_attention_args* args, void* workspace, size_t workspace_bytes,
                                           void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FLARE_OPS_H_ */
