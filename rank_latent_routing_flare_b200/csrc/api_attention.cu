// Host entry points of the exact softmax attention (include/flare_ops.h):
// argument checks before anything is enqueued, the choice of kernel and of
// the split along the keys, the workspace layout and the launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "attention.h"
#include "flare_ops.h"
#include "host_internal.h"
#include "ops_internal.h"

namespace flare {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();   // api.cu

namespace {

// Sizes the kernels cover; depends on the sizes alone, as the plan does, so a
// given problem always takes the same kernels and gives the same bits.
flare_status check_sizes(int64_t B, int64_t Hq, int64_t Hk, int64_t Nq, int64_t Nk, int64_t D) {
  if (B < 1 || Hq < 1 || Hk < 1 || Nq < 1 || Nk < 1 || Hq % Hk != 0) return FLARE_ERR_SHAPE;
  if (!row_width_ok(D)) return FLARE_ERR_UNSUPPORTED;
  constexpr int64_t most = int64_t(1) << 27;   // a query tile of a CTA waits for the keys of the other: half a second at most
  if (Nq > most || Nk > most || B > 65535 || Hq > 65535) return FLARE_ERR_UNSUPPORTED;
  // a CTA has eight rows of a head at least
  if (B * Hq * ((Nq + 7) / 8) > kMaxInt || B * Hk * ((Nk + 127) / 128) > kMaxInt) return FLARE_ERR_UNSUPPORTED;
  return FLARE_OK;
}

struct AttnPlan {
  bool step;           // few rows: attn_step
  int splits;
  int row_blocks;      // backward
  size_t off_doc, off_part_o, off_part_l, off_rows, total;
};

AttnPlan make_attn_plan(int64_t B, int64_t Hq, int64_t Hk, int64_t Nq, int64_t Nk, int64_t D, bool backward) {
  AttnPlan pl{};
  pl.step = Hq / Hk * Nq <= kAttnStepRows;
  if (pl.step) {
    // CTAs for two waves: few enough that their beginnings and ends do not
    // show, many enough that ragged caches even out; up to four while a split
    // has 2048 keys.  With two (three, four) waves, D = 128, 8 key heads: 64 ragged
    // caches of 1024 keys 31 us (34, 38), 16 of 8192 63 (64, 64), 16 of 32768 203
    // (198, 194).  Eight splits join in their cluster; more, in a launch of 5 us,
    // have 512 keys each.
    const int64_t wave = kNumSM * attn_step_ctas(static_cast<int>(D)), heads = B * Hk;
    const int64_t want = std::max(2 * wave / heads, std::min(4 * wave / heads, Nk / 2048));
    const int64_t most = std::max(std::min<int64_t>(Nk / 128, kAttnClusterSplits), Nk / 512);
    pl.splits = static_cast<int>(std::max<int64_t>(1, std::min({want, most, int64_t(256)})));
  } else {
    // one CTA per 256 rows of a head; where those leave half of the GPU idle,
    // the keys are split until they fill it, four key tiles a split at least
    const int64_t ctas = cdiv(Nq, 2 * kAttnQTile) * B * Hq, slots = kNumSM * (D == 128 ? 1 : 2);
    const int64_t tiles = cdiv(Nk, D == 128 ? 128 : 64);
    pl.splits = ctas * 2 > slots ? 1 : static_cast<int>(std::max<int64_t>(1, std::min(slots / ctas, tiles / 4)));
  }
  size_t off = 256;   // error word
  pl.off_doc = off;
  off += align256(static_cast<size_t>(B * Nk) * sizeof(int2));
  const size_t rows = static_cast<size_t>(B * Hq * Nq);
  if (backward) {
    const int64_t t = attn_bwd_stream_tile(static_cast<int>(D), true);
    pl.row_blocks = static_cast<int>(cdiv(Nq, t));
    pl.off_rows = off;
    off += align256(static_cast<size_t>(B * Hq) * pl.row_blocks * t * kAttnRowFields * 4);
  } else if (pl.splits > kAttnClusterSplits) {
    pl.off_part_o = off;
    off += align256(rows * pl.splits * D * 4);
    pl.off_part_l = off;
    off += align256(rows * pl.splits * 4);
  }
  pl.total = off;
  return pl;
}

// 4-D map of [B][H][N][D] rows: box of `rows` rows of one panel (up to 64
// elements) of one head, in the swizzle of that panel's width.
bool map_rows(CUtensorMap* m, const void* base, const long (&st)[3], int64_t B, int64_t H, int64_t N, int64_t D, int rows) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  const int64_t panel = std::min<int64_t>(D, 64);
  const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(N), cuuint64_t(H), cuuint64_t(B)};
  const cuuint64_t any = cuuint64_t(D) * 2;   // of a dimension of size one
  const cuuint64_t strides[3] = {N > 1 ? cuuint64_t(st[2]) * 2 : any, H > 1 ? cuuint64_t(st[1]) * 2 : any,
                                 B > 1 ? cuuint64_t(st[0]) * 2 : any};
  const cuuint32_t box[4] = {cuuint32_t(panel), cuuint32_t(rows), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle sw = panel == 16   ? CU_TENSOR_MAP_SWIZZLE_32B
                                : panel == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                              : CU_TENSOR_MAP_SWIZZLE_128B;
  auto encode = [&] {
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  // a thread that has made no CUDA call yet (a backward's) has no context
  // current, which setting its device mends (during a capture too)
  int dev;
  return encode() || (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode());
}

// Rows that TMA reads: no broadcast (zero stride).
flare_status tma_strides(long (&out)[3], const void* base, const int64_t* s, int64_t B, int64_t H, int64_t N, int64_t D) {
  const flare_status r = fill_strides(out, base, s, B, H, N, D, false);
  if (r != FLARE_OK) return r;
  if ((B > 1 && out[0] == 0) || (H > 1 && out[1] == 0) || (N > 1 && out[2] == 0)) return FLARE_ERR_UNSUPPORTED;
  return FLARE_OK;
}

struct Rows {
  long q[3], k[3], v[3];
};

flare_status fill_common(const flare_attention_args* a, bool backward, const void* ws, size_t ws_bytes, AttnPlan* pl,
                         AttnParams* p, Rows* r) {
  flare_status st = check_sizes(a->B, a->Hq, a->Hk, a->Nq, a->Nk, a->D);
  if (st != FLARE_OK) return st;
  if (!a->Q || !a->K || !a->V || !a->Y || !ws) return FLARE_ERR_NULL;
  if (a->prefix && !a->causal) return FLARE_ERR_SHAPE;
  if (!std::isfinite(a->scale) || !std::isfinite(a->cap)) return FLARE_ERR_SHAPE;
  if (a->scale > 0.0 && (a->scale < 1e-30 || a->scale > 1e30)) return FLARE_ERR_UNSUPPORTED;   // what fp32 holds with room for products
  if (a->cap > 0.0 && (a->cap < 1e-6 || a->cap > 1e9)) return FLARE_ERR_UNSUPPORTED;   // what the tanh is accurate for
  st = tma_strides(r->q, a->Q, a->q_stride, a->B, a->Hq, a->Nq, a->D);
  if (st == FLARE_OK) st = tma_strides(r->k, a->K, a->k_stride, a->B, a->Hk, a->Nk, a->D);
  if (st == FLARE_OK) st = tma_strides(r->v, a->V, a->v_stride, a->B, a->Hk, a->Nk, a->D);
  if (st != FLARE_OK) return st;
  for (const void* q : {static_cast<const void*>(a->lengths), static_cast<const void*>(a->q_lengths),
                        static_cast<const void*>(a->q_offsets), static_cast<const void*>(a->documents),
                        static_cast<const void*>(a->prefix), static_cast<const void*>(a->slopes),
                        static_cast<const void*>(a->L)})
    if (!aligned4(q)) return FLARE_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(ws) % 256 != 0) return FLARE_ERR_ALIGN;
  *pl = make_attn_plan(a->B, a->Hq, a->Hk, a->Nq, a->Nk, a->D, backward);
  if (ws_bytes < pl->total) return FLARE_ERR_WORKSPACE;
  uint8_t* w = static_cast<uint8_t*>(const_cast<void*>(ws));
  *p = AttnParams{};
  p->B = static_cast<int>(a->B);
  p->Hq = static_cast<int>(a->Hq);
  p->Hk = static_cast<int>(a->Hk);
  p->G = static_cast<int>(a->Hq / a->Hk);
  p->D = static_cast<int>(a->D);
  p->mask = AttnMask{static_cast<int>(a->Nq), static_cast<int>(a->Nk), a->causal ? 1 : 0, a->lengths, a->q_lengths,
                     a->q_offsets, a->prefix, a->documents ? reinterpret_cast<const int2*>(w + pl->off_doc) : nullptr};
  p->scale = resolve_scale(static_cast<float>(a->scale), p->D);
  p->cap = a->cap > 0.0 ? static_cast<float>(a->cap) : 0.f;
  p->slopes = a->slopes;
  p->L = a->L;
  p->splits = pl->splits;
  p->err = reinterpret_cast<uint32_t*>(w);
  p->timeout_ns = wait_timeout_ns();
  return FLARE_OK;
}

bool documents(const flare_attention_args* a, const AttnPlan& pl, void* ws, cudaStream_t s) {
  if (!a->documents) return true;
  return launch_attn_documents(a->documents, reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + pl.off_doc),
                               static_cast<int>(a->B), static_cast<int>(a->Nk), s) == cudaSuccess;
}

}  // namespace
}  // namespace flare

using namespace flare;

extern "C" {

size_t flare_attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Hk, int64_t Nq, int64_t Nk, int64_t D,
                                       int backward) {
  if (check_sizes(B, Hq, Hk, Nq, Nk, D) != FLARE_OK) return 0;
  return make_attn_plan(B, Hq, Hk, Nq, Nk, D, backward != 0).total;
}

flare_status flare_attention_fwd(const flare_attention_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  if (!a) return FLARE_ERR_NULL;
  AttnPlan pl;
  AttnParams p;
  Rows r;
  flare_status st = fill_common(a, false, workspace, workspace_bytes, &pl, &p, &r);
  if (st != FLARE_OK) return st;
  st = fill_strides(p.ys, a->Y, a->y_stride, a->B, a->Hq, a->Nq, a->D, true);
  if (st != FLARE_OK) return st;
  p.y = a->Y;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(w + pl.off_part_o);
  p.part_l = reinterpret_cast<float*>(w + pl.off_part_l);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!documents(a, pl, workspace, s)) return FLARE_ERR_LAUNCH;
  if (pl.step) {
    const AttnSide q{a->Q, r.q[0], r.q[1], r.q[2]}, k{a->K, r.k[0], r.k[1], r.k[2]}, v{a->V, r.v[0], r.v[1], r.v[2]};
    if (launch_attn_step(p, q, k, v, s) != cudaSuccess) return FLARE_ERR_LAUNCH;
  } else {
    AttnMaps m;
    const int kt = attn_fwd_key_tile(p.D, p.slopes != nullptr, p.cap > 0.f);
    if (!map_rows(&m.q, a->Q, r.q, a->B, a->Hq, a->Nq, a->D, kAttnQTile) ||
        !map_rows(&m.k, a->K, r.k, a->B, a->Hk, a->Nk, a->D, kt) || !map_rows(&m.v, a->V, r.v, a->B, a->Hk, a->Nk, a->D, kt))
      return FLARE_ERR_LAUNCH;
    if (launch_attn_fwd(m, p, s) != cudaSuccess) return FLARE_ERR_LAUNCH;
  }
  if (p.splits > kAttnClusterSplits && launch_attn_join(p, s) != cudaSuccess) return FLARE_ERR_LAUNCH;
  return FLARE_OK;
}

flare_status flare_attention_bwd(const flare_attention_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  if (!a) return FLARE_ERR_NULL;
  AttnPlan pl;
  AttnBwdParams p{};
  Rows r;
  flare_status st = fill_common(a, true, workspace, workspace_bytes, &pl, &p.a, &r);
  if (st != FLARE_OK) return st;
  if (!a->L || !a->dY || !a->dQ || !a->dK || !a->dV) return FLARE_ERR_NULL;
  long ys[3], dys[3];
  st = fill_strides(ys, a->Y, a->y_stride, a->B, a->Hq, a->Nq, a->D, false);
  if (st == FLARE_OK) st = tma_strides(dys, a->dY, a->dy_stride, a->B, a->Hq, a->Nq, a->D);
  if (st == FLARE_OK) st = fill_strides(p.dqs, a->dQ, a->dq_stride, a->B, a->Hq, a->Nq, a->D, true);
  if (st == FLARE_OK) st = fill_strides(p.dks, a->dK, a->dk_stride, a->B, a->Hk, a->Nk, a->D, true);
  if (st == FLARE_OK) st = fill_strides(p.dvs, a->dV, a->dv_stride, a->B, a->Hk, a->Nk, a->D, true);
  if (st != FLARE_OK) return st;
  p.q = AttnSide{a->Q, r.q[0], r.q[1], r.q[2]};
  p.k = AttnSide{a->K, r.k[0], r.k[1], r.k[2]};
  p.v = AttnSide{a->V, r.v[0], r.v[1], r.v[2]};
  p.yin = AttnSide{a->Y, ys[0], ys[1], ys[2]};
  p.dy = AttnSide{a->dY, dys[0], dys[1], dys[2]};
  p.dq = a->dQ;
  p.dk = a->dK;
  p.dv = a->dV;
  p.rows = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.off_rows);
  p.row_blocks = pl.row_blocks;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!documents(a, pl, workspace, s) || launch_attn_rows(p, s) != cudaSuccess) return FLARE_ERR_LAUNCH;
  // the dQ pass keeps tiles of 128 rows of Q and dY and streams K and V; the dK/dV pass the other way round
  const int tq = attn_bwd_stream_tile(p.a.D, false), tkv = attn_bwd_stream_tile(p.a.D, true);
  AttnMaps dq, dkv;
  // a pass that keeps its own tile of rows in TMEM reads it without a map (any map stands in)
  bool ok = map_rows(&dq.k, a->K, r.k, a->B, a->Hk, a->Nk, a->D, tq) && map_rows(&dq.v, a->V, r.v, a->B, a->Hk, a->Nk, a->D, tq) &&
            map_rows(&dkv.q, a->Q, r.q, a->B, a->Hq, a->Nq, a->D, tkv) && map_rows(&dkv.dy, a->dY, dys, a->B, a->Hq, a->Nq, a->D, tkv);
  dq.q = dq.k;
  dq.dy = dq.v;
  if (!attn_bwd_rows_in_tmem(p.a.D, false))
    ok = ok && map_rows(&dq.q, a->Q, r.q, a->B, a->Hq, a->Nq, a->D, 128) && map_rows(&dq.dy, a->dY, dys, a->B, a->Hq, a->Nq, a->D, 128);
  dkv.k = dkv.q;
  dkv.v = dkv.dy;
  if (!attn_bwd_rows_in_tmem(p.a.D, true))
    ok = ok && map_rows(&dkv.k, a->K, r.k, a->B, a->Hk, a->Nk, a->D, 128) && map_rows(&dkv.v, a->V, r.v, a->B, a->Hk, a->Nk, a->D, 128);
  if (!ok) return FLARE_ERR_LAUNCH;
  if (launch_attn_bwd_dq(dq, p, s) != cudaSuccess || launch_attn_bwd_dkv(dkv, p, s) != cudaSuccess)
    return FLARE_ERR_LAUNCH;
  return FLARE_OK;
}

}  // extern "C"
