// Host entry points of the query/key preparation (include/flare_ops.h):
// argument checks, before anything is enqueued, and the launches.
#include "flare_ops.h"
#include "host_internal.h"
#include "norm_rope.h"
#include "ops_internal.h"

namespace flare {
namespace {

// Sizes the kernels cover.  32768 columns: every CTA leaves a partial row of
// the gains' gradients, 40 MB of workspace for two CTAs an SM.
flare_status check_sizes(int64_t B, int64_t N, int64_t Hq, int64_t Hk, int64_t D) {
  if (B < 1 || N < 1 || Hq < 0 || Hk < 0 || Hq + Hk < 1) return FLARE_ERR_SHAPE;
  if (!row_width_ok(D)) return FLARE_ERR_UNSUPPORTED;
  if (N > kMaxInt || B > kMaxInt || Hq > 32768 || Hk > 32768 || (Hq + Hk) * D > 32768) return FLARE_ERR_UNSUPPORTED;
  if (B > (int64_t(1) << 40) / N || B * N > kMaxInt) return FLARE_ERR_UNSUPPORTED;
  return FLARE_OK;
}

// One of the two tensors; out: the forward's output or the backward's dx.
flare_status fill_side(NormRopeSide* s, int64_t B, int64_t N, int64_t D, int64_t H, const flare_bf16* x,
                       const int64_t* xs, const float* gain, int64_t per_head, const flare_bf16* dy,
                       const int64_t* ds, flare_bf16* out, const int64_t* os, float* dgain, bool backward) {
  *s = NormRopeSide{};
  if (H == 0) return x || gain || dy || out || dgain ? FLARE_ERR_SHAPE : FLARE_OK;
  if (!x || !out || (backward && !dy)) return FLARE_ERR_NULL;
  if (dgain && !gain) return FLARE_ERR_NULL;
  s->H = static_cast<int>(H);
  s->gain_per_head = per_head ? 1 : 0;
  s->x = x;
  s->dy = dy;
  s->y = out;
  s->gain = gain;
  s->dgain = dgain;
  flare_status r = fill_strides(s->xs, x, xs, B, H, N, D, false);
  if (r == FLARE_OK) r = fill_strides(s->ys, out, os, B, H, N, D, true);
  if (r == FLARE_OK && backward) r = fill_strides(s->ds, dy, ds, B, H, N, D, false);
  if (r == FLARE_OK && (!aligned16(gain) || !aligned16(dgain))) r = FLARE_ERR_ALIGN;
  return r;
}

flare_status fill(const flare_qk_norm_rope_args* a, bool backward, NormRopeParams* p) {
  *p = NormRopeParams{};
  flare_status r = check_sizes(a->B, a->N, a->Hq, a->Hk, a->D);
  if (r != FLARE_OK) return r;
  if (a->rot < 0 || a->rot > a->D || a->rot % 2 != 0 || !(a->eps >= 0.0)) return FLARE_ERR_SHAPE;
  if (!a->interleaved && a->rot % 16 != 0) return FLARE_ERR_UNSUPPORTED;
  if (a->rot > 0) {
    if (!a->freqs) return FLARE_ERR_NULL;
    if (a->pos_kind < 0 || a->pos_kind > 2) return FLARE_ERR_SHAPE;
    if (a->axes < 1 || a->axes > 4 || (a->pos_kind != 2 && a->axes != 1)) return FLARE_ERR_SHAPE;
    if ((a->pos_kind != 0) != (a->positions != nullptr)) return FLARE_ERR_NULL;
  } else if (a->freqs || a->positions) {
    return FLARE_ERR_SHAPE;
  }
  if (!aligned4(a->freqs) || !aligned4(a->positions) || !aligned4(a->lengths)) return FLARE_ERR_ALIGN;
  p->B = static_cast<int>(a->B);
  p->N = static_cast<int>(a->N);
  p->D = static_cast<int>(a->D);
  p->P = static_cast<int>(a->rot / 2);
  p->axes = static_cast<int>(a->axes);
  p->pos_kind = static_cast<int>(a->pos_kind);
  p->interleaved = a->interleaved ? 1 : 0;
  p->freqs = a->freqs;
  p->pos = a->positions;
  p->lengths = a->lengths;
  p->eps = static_cast<float>(a->eps);
  r = fill_side(&p->side[0], a->B, a->N, a->D, a->Hq, a->Q, a->q_stride, a->q_gain, a->q_gain_per_head, backward ? a->Qr : nullptr,
                a->qr_stride, backward ? a->dQ : a->Qr, backward ? a->dq_stride : a->qr_stride,
                backward ? a->dq_gain : nullptr, backward);
  if (r != FLARE_OK) return r;
  r = fill_side(&p->side[1], a->B, a->N, a->D, a->Hk, a->K, a->k_stride, a->k_gain, a->k_gain_per_head, backward ? a->Kr : nullptr,
                a->kr_stride, backward ? a->dK : a->Kr, backward ? a->dk_stride : a->kr_stride,
                backward ? a->dk_gain : nullptr, backward);
  if (r != FLARE_OK) return r;
  norm_rope_plan(p);
  return FLARE_OK;
}

}  // namespace
}  // namespace flare

using namespace flare;

extern "C" {

size_t flare_qk_norm_rope_workspace_bytes(int64_t B, int64_t N, int64_t Hq, int64_t Hk, int64_t D) {
  if (check_sizes(B, N, Hq, Hk, D) != FLARE_OK) return 0;
  return align256(norm_rope_part_floats(B, N, Hq, Hk, D) * sizeof(float));
}

flare_status flare_qk_norm_rope_fwd(const flare_qk_norm_rope_args* args, void* stream) {
  if (!args) return FLARE_ERR_NULL;
  NormRopeParams p;
  const flare_status r = fill(args, false, &p);
  if (r != FLARE_OK) return r;
  return launch_norm_rope_fwd(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FLARE_OK : FLARE_ERR_LAUNCH;
}

flare_status flare_qk_norm_rope_bwd(const flare_qk_norm_rope_args* args, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  if (!args) return FLARE_ERR_NULL;
  NormRopeParams p;
  const flare_status r = fill(args, true, &p);
  if (r != FLARE_OK) return r;
  if (p.side[0].dgain || p.side[1].dgain) {
    if (!workspace) return FLARE_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return FLARE_ERR_ALIGN;
    if (workspace_bytes < flare_qk_norm_rope_workspace_bytes(args->B, args->N, args->Hq, args->Hk, args->D))
      return FLARE_ERR_WORKSPACE;
    p.part = static_cast<float*>(workspace);
  }
  return launch_norm_rope_bwd(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FLARE_OK : FLARE_ERR_LAUNCH;
}

}  // extern "C"
