// kv8_abi.cu -- the extern "C" entry points of the 8-bit KV cache path
// (include/csa.h): argument validation before any launch.
#include <cmath>

#include "common.cuh"
#include "kv8.h"

namespace csa {

static bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static cudaStream_t S(csa_stream_t s) { return (cudaStream_t)s; }

static csa_status check_rope(const csa_rope* r) {
  if (r == nullptr) return CSA_ERR_ARG;
  if (r->d <= 0 || r->d % 8 != 0 || r->d > 512) return CSA_ERR_SHAPE;
  if (r->rope_dims < 0 || (r->rope_dims & 1) || r->rope_off < 0 || r->rope_dims > r->d ||
      r->rope_off > r->d - r->rope_dims)
    return CSA_ERR_SHAPE;
  if (r->layout != CSA_ROPE_INTERLEAVED && r->layout != CSA_ROPE_HALF) return CSA_ERR_ARG;
  if (!std::isfinite(r->mscale)) return CSA_ERR_ARG;
  return CSA_OK;
}

static csa_status check_kv8(const csa_kv8_params* p) {
  if (p == nullptr) return CSA_ERR_ARG;
  if (p->n_q <= 0 || p->n_kv <= 0 || p->n_q % p->n_kv != 0) return CSA_ERR_SHAPE;
  if (p->block != 16 && p->block != 32 && p->block != 64 && p->block != 128) return CSA_ERR_SHAPE;
  if (p->N <= 0 || p->N % p->block != 0) return CSA_ERR_SHAPE;
  if (p->d != 64 && p->d != 128 && p->d != 256) return CSA_ERR_UNSUPPORTED;
  if (p->act != CSA_F32 && p->act != CSA_BF16) return CSA_ERR_DTYPE;
  return CSA_OK;
}

static csa_status check_cache(const void* kc, const uint8_t* k_exp, const void* vc,
                              const uint8_t* v_exp) {
  if (!kc || !k_exp || !vc || !v_exp) return CSA_ERR_ARG;
  return aligned16(kc) && aligned16(vc) ? CSA_OK : CSA_ERR_ALIGN;
}

}  // namespace csa

using namespace csa;

extern "C" {

csa_status csa_rope_freqs(const csa_rope* r, double* turns, csa_stream_t stream) {
  csa_status st = check_rope(r);
  if (st != CSA_OK) return st;
  if (!(r->base > 0.f) || !std::isfinite(r->base)) return CSA_ERR_ARG;
  if (r->scaling < CSA_ROPE_NONE || r->scaling > CSA_ROPE_PARTS) return CSA_ERR_ARG;
  if (r->scaling != CSA_ROPE_NONE && (!(r->factor > 0.f) || !std::isfinite(r->factor)))
    return CSA_ERR_ARG;
  if (r->scaling == CSA_ROPE_PARTS &&
      (!(r->orig_len > 0.f) || !(r->fast > r->slow) || !std::isfinite(r->orig_len) ||
       !std::isfinite(r->fast) || !std::isfinite(r->slow)))
    return CSA_ERR_ARG;
  if (r->rope_dims == 0) return CSA_OK;
  if (!turns) return CSA_ERR_ARG;
  if ((uintptr_t)turns & 7u) return CSA_ERR_ALIGN;
  return launch_rope_freqs(*r, turns, S(stream));
}

csa_status csa_qk_norm_rope(const csa_rope* r, int R, int n_q, int n_kv, int act, int norm,
                            float eps, const double* turns, const int32_t* pos, const void* q,
                            int64_t q_stride, const float* q_gain, const void* k,
                            int64_t k_stride, const float* k_gain, void* q_out,
                            int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                            csa_stream_t stream) {
  csa_status st = check_rope(r);
  if (st != CSA_OK) return st;
  if (act != CSA_F32 && act != CSA_BF16) return CSA_ERR_DTYPE;
  if (norm != 0 && norm != 1) return CSA_ERR_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return CSA_ERR_ARG;
  if (R < 0 || n_q <= 0 || n_kv < 0 || n_q > 65535 || n_kv > 65535) return CSA_ERR_SHAPE;
  const int64_t es = act == CSA_F32 ? 4 : 2;
  const int64_t strides[4] = {q_stride, q_out_stride, k_stride, k_out_stride};
  for (int i = 0; i < (n_kv ? 4 : 2); ++i) {
    if (strides[i] < (int64_t)(i < 2 ? n_q : n_kv) * r->d) return CSA_ERR_SHAPE;
    if (strides[i] * es % 16 != 0) return CSA_ERR_ALIGN;
  }
  if (R == 0) return CSA_OK;
  if (!pos || !q || !q_out || (n_kv > 0) != (k != nullptr) || (n_kv > 0) != (k_out != nullptr))
    return CSA_ERR_ARG;
  if (r->rope_dims > 0 && !turns) return CSA_ERR_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned16(q_gain) || !aligned16(k_gain) || ((uintptr_t)turns & 7u) || ((uintptr_t)pos & 3u))
    return CSA_ERR_ALIGN;
  NormRopeArgs a;
  a.turns = turns; a.pos = pos;
  a.x[0] = q; a.x[1] = k;
  a.out[0] = q_out; a.out[1] = k_out;
  a.gain[0] = q_gain; a.gain[1] = k_gain;
  a.stride[0] = q_stride; a.stride[1] = k_stride;
  a.out_stride[0] = q_out_stride; a.out_stride[1] = k_out_stride;
  a.heads[0] = n_q; a.heads[1] = n_kv;
  a.d = r->d; a.rope_dims = r->rope_dims; a.rope_off = r->rope_off;
  a.half = r->layout == CSA_ROPE_HALF;
  a.norm = norm;
  a.eps = eps; a.mscale = r->mscale;
  return launch_qk_norm_rope(a, R, act, S(stream));
}

csa_status csa_kv8_append(const csa_kv8_params* p, int B, int T, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const int32_t* n_old,
                          const int32_t* n_new, void* kc, uint8_t* k_exp, void* vc,
                          uint8_t* v_exp, csa_stream_t stream) {
  csa_status st = check_kv8(p);
  if (st != CSA_OK) return st;
  if (B <= 0 || T < 0) return CSA_ERR_SHAPE;
  const int64_t es = p->act == CSA_F32 ? 4 : 2, row = (int64_t)p->n_kv * p->d;
  if (k_stride < row || v_stride < row) return CSA_ERR_SHAPE;
  if (k_stride * es % 16 != 0 || v_stride * es % 16 != 0) return CSA_ERR_ALIGN;
  if (T == 0) return CSA_OK;
  if (!k || !v || !n_old) return CSA_ERR_ARG;
  st = check_cache(kc, k_exp, vc, v_exp);
  if (st != CSA_OK) return st;
  if (!aligned16(k) || !aligned16(v) || ((uintptr_t)n_old & 3u) || ((uintptr_t)n_new & 3u))
    return CSA_ERR_ALIGN;
  return launch_kv8_append(*p, B, T, k, k_stride, v, v_stride, n_old, n_new,
                           Kv8Cache{(uint8_t*)kc, k_exp, (uint8_t*)vc, v_exp}, S(stream));
}

size_t csa_kv8_attend_workspace_bytes(const csa_kv8_params* p, int B, int Q, int with_acc) {
  if (check_kv8(p) != CSA_OK || B <= 0 || Q <= 0) return 0;
  return kv8_attend_ws_bytes(*p, B, Q, with_acc != 0);
}

csa_status csa_kv8_attend(const csa_kv8_params* p, int B, int Q, float scale, const void* q,
                          const int32_t* n_vis, const void* kc, const uint8_t* k_exp,
                          const void* vc, const uint8_t* v_exp, const float* sink, void* out,
                          float* acc, float decay, void* workspace, size_t ws_bytes,
                          csa_stream_t stream) {
  csa_status st = check_kv8(p);
  if (st != CSA_OK) return st;
  if (B <= 0 || Q <= 0) return CSA_ERR_SHAPE;
  if (!std::isfinite(scale) || (acc && !std::isfinite(decay))) return CSA_ERR_ARG;
  if (!q || !n_vis || !out) return CSA_ERR_ARG;
  st = check_cache(kc, k_exp, vc, v_exp);
  if (st != CSA_OK) return st;
  if (!aligned16(q) || !aligned16(out) || ((uintptr_t)n_vis & 3u) || ((uintptr_t)sink & 3u) ||
      ((uintptr_t)acc & 3u))
    return CSA_ERR_ALIGN;
  const size_t need = kv8_attend_ws_bytes(*p, B, Q, acc != nullptr);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return CSA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return CSA_ERR_ALIGN;
  return launch_kv8_attend(*p, B, Q, scale, q, n_vis,
                           Kv8Cache{(uint8_t*)kc, (uint8_t*)k_exp, (uint8_t*)vc, (uint8_t*)v_exp},
                           sink, out, acc, decay, workspace, S(stream));
}

csa_status csa_kv8_evict(const csa_kv8_params* p, int B, int keep, int recent, const float* acc,
                         const int32_t* n_tok, void* kc, uint8_t* k_exp, void* vc,
                         uint8_t* v_exp, int32_t* kept, float* acc_out, int32_t* n_tok_out,
                         csa_stream_t stream) {
  csa_status st = check_kv8(p);
  if (st != CSA_OK) return st;
  if (B <= 0) return CSA_ERR_SHAPE;
  const int NB = p->N / p->block;
  if (recent < 1 || recent > keep || keep > NB) return CSA_ERR_SHAPE;
  if (NB > kKv8MaxBlocks) return CSA_ERR_UNSUPPORTED;
  if (!acc || !n_tok || !kept || !acc_out || !n_tok_out) return CSA_ERR_ARG;
  st = check_cache(kc, k_exp, vc, v_exp);
  if (st != CSA_OK) return st;
  if (((uintptr_t)acc & 3u) || ((uintptr_t)n_tok & 3u) || ((uintptr_t)kept & 3u) ||
      ((uintptr_t)acc_out & 3u) || ((uintptr_t)n_tok_out & 3u))
    return CSA_ERR_ALIGN;
  return launch_kv8_evict(*p, B, keep, recent, acc, n_tok,
                          Kv8Cache{(uint8_t*)kc, k_exp, (uint8_t*)vc, v_exp}, kept, acc_out,
                          n_tok_out, S(stream));
}

}  // extern "C"
