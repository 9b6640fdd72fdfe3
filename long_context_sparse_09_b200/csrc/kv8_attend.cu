// kv8_attend.cu -- grouped-query attention over the 8-bit KV cache
// (csa_kv8_attend).
//
// Simple form: a CTA owns one query row and head.  It walks the visible slots
// in tiles of one per thread with a running maximum and sum (base 2), a
// thread scoring a slot and then summing p * value for its dims.  For the
// accumulated weights it notes the log2 of every block's weight sum and of
// the row's denominator; kv8_acc adds them up in a fixed order.
#include "common.cuh"
#include "kv8.h"

namespace csa {

namespace {

constexpr int kSimpleThreads = 128;
constexpr int kAccThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

struct Kv8AttnArgs {
  const void* q;
  const int32_t* n_vis;
  Kv8Cache c;
  const float* sink;
  void* out;
  float* blk_log;   // [B][H][Q G][NB] log2 of each block's weight sum (unnormalised)
  float* row_log;   // [B][H][Q G] log2 of the row's denominator
  float* acc;
  unsigned* err;
  int B, Q, H, G, d, N, NB, block;
  float scale2, decay;  // softmax scale times log2(e)
};

__device__ __forceinline__ float pow2e8(uint8_t e) {
  return __int_as_float(max((int)e, 1) << 23);
}

template <typename T>
__global__ void __launch_bounds__(kSimpleThreads) kv8_attend_simple(Kv8AttnArgs a) {
  __shared__ float qs[256], ps[kSimpleThreads], red[32];
  pdl_wait();
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / (a.H * a.G);  // b Q + j
  const int hq = (int)(blockIdx.x % (a.H * a.G)), h = hq / a.G, b = (int)(row / a.Q);
  int n = a.n_vis[row];
  if (n > a.N && tid == 0) atomicOr(a.err, CSA_DEV_BAD_INDEX);
  n = min(max(n, 0), a.N);
  const T* q = reinterpret_cast<const T*>(a.q) + (row * a.H * a.G + hq) * a.d;
  for (int i = tid; i < a.d; i += kSimpleThreads) qs[i] = to_f32(q[i]) * a.scale2;
  __syncthreads();
  const int64_t head = (int64_t)b * a.H + h;
  const int64_t lrow = head * a.Q * a.G + (int64_t)(row % a.Q) * a.G + hq % a.G;
  const uint8_t* kc = a.c.kc + head * a.N * a.d;
  const uint8_t* vc = a.c.vc + head * a.N * a.d;
  float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
  for (int s0 = 0; s0 < n; s0 += kSimpleThreads) {
    const int s = s0 + tid;
    float x = -INFINITY;
    if (s < n) {
      x = 0.f;
      for (int i = 0; i < a.d; ++i) x = fmaf(qs[i], e4m3_to_f32(kc[(int64_t)s * a.d + i]), x);
      x *= pow2e8(a.c.k_exp[head * a.NB + s / a.block]);
    }
    const float m1 = fmaxf(m, block_reduce<true>(x, red));
    const float p = s < n ? exp2f(x - m1) : 0.f, f = exp2f(m - m1);
    ps[tid] = p;
    l = l * f + block_reduce<false>(p, red);
    if (a.blk_log && tid * a.block < kSimpleThreads && s0 + tid * a.block < n) {
      float t = 0.f;
      for (int i = 0; i < a.block; ++i) t += ps[tid * a.block + i];
      a.blk_log[lrow * a.NB + s0 / a.block + tid] = log2f(t) + m1;
    }
    for (int k = 0; k < 2; ++k) {
      const int i = tid + k * kSimpleThreads;
      o[k] *= f;
      if (i < a.d)
        for (int t = 0; t < min(kSimpleThreads, n - s0); ++t)
          o[k] = fmaf(ps[t] * pow2e8(a.c.v_exp[head * a.NB + (s0 + t) / a.block]),
                      e4m3_to_f32(vc[(int64_t)(s0 + t) * a.d + i]), o[k]);
    }
    m = m1;
    __syncthreads();
  }
  if (a.sink && n > 0) {
    const float z = a.sink[hq] * kLog2e, m1 = fmaxf(m, z), f = exp2f(m - m1);
    l = l * f + exp2f(z - m1);
    o[0] *= f;
    o[1] *= f;
    m = m1;
  }
  if (a.row_log && tid == 0) a.row_log[lrow] = n > 0 ? log2f(l) + m : 0.f;
  T* out = reinterpret_cast<T*>(a.out) + (row * a.H * a.G + hq) * a.d;
  for (int k = 0; k < 2; ++k) {
    const int i = tid + k * kSimpleThreads;
    if (i < a.d) out[i] = from_f32<T>(n > 0 ? o[k] / l : 0.f);
  }
}

__global__ void __launch_bounds__(kAccThreads) kv8_acc_kernel(Kv8AttnArgs a, int tiles) {
  pdl_wait();
  const int64_t head = blockIdx.x / tiles;
  const int i = (int)(blockIdx.x % tiles) * kAccThreads + threadIdx.x;
  if (i >= a.NB) return;
  const int b = (int)(head / a.H);
  float sum = 0.f;
  bool seen = false;
  for (int j = 0; j < a.Q; ++j) {
    if ((int64_t)i * a.block >= min(a.n_vis[(int64_t)b * a.Q + j], a.N)) continue;
    seen = true;
    for (int g = 0; g < a.G; ++g) {
      const int64_t lrow = (head * a.Q + j) * a.G + g;
      sum += exp2f(a.blk_log[lrow * a.NB + i] - a.row_log[lrow]);
    }
  }
  if (!seen) return;
  float* acc = a.acc + head * a.NB + i;
  *acc = a.decay == 0.f ? sum : fmaf(a.decay, *acc, sum);
}

}  // namespace

size_t kv8_attend_ws_bytes(const csa_kv8_params& p, int B, int Q, bool acc) {
  const size_t rows = (size_t)B * Q * p.n_q;
  return acc ? align_up(rows * (p.N / p.block) * 4, 256) + align_up(rows * 4, 256) : 0;
}

csa_status launch_kv8_attend(const csa_kv8_params& p, int B, int Q, float scale, const void* q,
                             const int32_t* n_vis, const Kv8Cache& c, const float* sink,
                             void* out, float* acc, float decay, void* ws, cudaStream_t st) {
  Kv8AttnArgs a = {};
  a.q = q; a.n_vis = n_vis; a.c = c; a.sink = sink; a.out = out;
  a.B = B; a.Q = Q; a.H = p.n_kv; a.G = p.n_q / p.n_kv; a.d = p.d; a.N = p.N;
  a.NB = p.N / p.block; a.block = p.block;
  a.scale2 = scale * kLog2e;
  a.decay = decay;
  a.err = device_error_word();
  if (a.err == nullptr) return CSA_ERR_CUDA;
  const size_t rows = (size_t)B * Q * p.n_q;
  if (acc) {
    a.acc = acc;
    a.blk_log = (float*)ws;
    a.row_log = (float*)((char*)ws + align_up(rows * a.NB * 4, 256));
  }
  if (rows > 0x7fffffff) return CSA_ERR_SHAPE;
  auto kern = p.act == CSA_F32 ? kv8_attend_simple<float> : kv8_attend_simple<__nv_bfloat16>;
  csa_status ok = CSA_OK;
  CSA_LAUNCH(KK_KV8_ATTEND, st,
             if (launch_maybe_pdl(true, kern, dim3((unsigned)rows), dim3(kSimpleThreads), 0, st,
                                  a) != cudaSuccess) ok = CSA_ERR_CUDA);
  if (acc) {
    const int tiles = (a.NB + kAccThreads - 1) / kAccThreads;
    CSA_LAUNCH(KK_KV8_ACC, st,
               if (launch_maybe_pdl(true, kv8_acc_kernel, dim3((unsigned)(B * a.H * tiles)),
                                    dim3(kAccThreads), 0, st, a, tiles) != cudaSuccess)
                 ok = CSA_ERR_CUDA);
  }
  return ok != CSA_OK ? ok : last_launch_status();
}

}  // namespace csa
