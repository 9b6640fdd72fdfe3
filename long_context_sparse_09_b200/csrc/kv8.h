// kv8.h -- host-side launchers of the 8-bit KV cache path (internal).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "csa.h"

namespace csa {

constexpr int kKv8MinExp = -110, kKv8MaxExp = 119;  // block exponents (include/csa.h)
constexpr int kKv8MaxBlocks = 262144;               // N / block that csa_kv8_evict ranks

// Codes and exponents of the K and V caches.
struct Kv8Cache {
  uint8_t* kc;
  uint8_t* k_exp;
  uint8_t* vc;
  uint8_t* v_exp;
};

csa_status launch_rope_freqs(const csa_rope& r, double* turns, cudaStream_t st);

struct NormRopeArgs {
  const double* turns;
  const int32_t* pos;
  const void* x[2];       // queries, keys
  void* out[2];
  const float* gain[2];
  int64_t stride[2], out_stride[2];  // elements between tokens
  int heads[2];
  int d, rope_dims, rope_off, half, norm;
  float eps, mscale;
};
csa_status launch_qk_norm_rope(const NormRopeArgs& a, int R, int act, cudaStream_t st);

csa_status launch_kv8_append(const csa_kv8_params& p, int B, int T, const void* k,
                             int64_t k_stride, const void* v, int64_t v_stride,
                             const int32_t* n_old, const int32_t* n_new, const Kv8Cache& c,
                             cudaStream_t st);

size_t kv8_attend_ws_bytes(const csa_kv8_params& p, int B, int Q, bool acc);
csa_status launch_kv8_attend(const csa_kv8_params& p, int B, int Q, float scale, const void* q,
                             const int32_t* n_vis, const Kv8Cache& c, const float* sink,
                             void* out, float* acc, float decay, void* ws, cudaStream_t st);

csa_status launch_kv8_evict(const csa_kv8_params& p, int B, int keep, int recent,
                            const float* acc, const int32_t* n_tok, const Kv8Cache& c,
                            int32_t* kept, float* acc_out, int32_t* n_tok_out, cudaStream_t st);

}  // namespace csa
