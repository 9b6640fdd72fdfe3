// kv8_rope.cu -- per-head RMSNorm and rotation of queries and keys in one
// pass (csa_qk_norm_rope), and the table of angles it reads.
//
//   y = x * gain / sqrt(mean(x^2) + eps);  (a, b) -> (a cos - b sin, a sin + b cos)
//
// A CTA owns one token: it forms the token's cos / sin once (fp64 turns,
// reduced to a fraction of a turn before fp32) and walks the token's heads,
// a group of lanes per head, 8 elements a lane and chunk.  The normalised row
// goes through shared memory, so a pair's partner may sit anywhere in it.
#include "common.cuh"
#include "kv8.h"

namespace csa {

namespace {

constexpr int kNrThreads = 256;

__global__ void rope_freqs_kernel(csa_rope r, double* __restrict__ turns) {
  const int p = blockIdx.x * blockDim.x + threadIdx.x;
  if (p >= r.rope_dims / 2) return;
  const double two_pi = 6.283185307179586476925286766559;
  double t = pow((double)r.base, -2.0 * p / r.rope_dims) / two_pi;
  if (r.scaling == CSA_ROPE_LINEAR) {
    t /= (double)r.factor;
  } else if (r.scaling == CSA_ROPE_PARTS) {
    double g = ((double)r.orig_len * t - r.slow) / ((double)r.fast - r.slow);
    g = fmin(fmax(g, 0.0), 1.0);
    t *= g + (1.0 - g) / (double)r.factor;
  }
  turns[p] = t;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// G lanes a head (a power of two, at least d / 8 up to 32), NC chunks a lane
// (2 only for d > 256).
template <typename T, int NC>
__global__ void __launch_bounds__(kNrThreads) qk_norm_rope_kernel(NormRopeArgs a, int G) {
  extern __shared__ float sm[];
  float2* cs = reinterpret_cast<float2*>(sm);         // [rope_dims / 2]
  float* rows = sm + 2 * (a.rope_dims / 2);           // [threads / G][d + 1]
  pdl_wait();
  const int64_t r = blockIdx.x;
  const int half_dims = a.rope_dims / 2;
  if (half_dims > 0) {
    const double pos = (double)a.pos[r];
    for (int p = threadIdx.x; p < half_dims; p += kNrThreads) {
      const double t = pos * a.turns[p];
      const float f = (float)(2.0 * (t - rint(t)));   // half turns in [-1, 1]
      float s, c;
      sincospif(f, &s, &c);
      cs[p] = make_float2(c * a.mscale, s * a.mscale);
    }
  }
  __syncthreads();
  const int per = kNrThreads / G, sub = threadIdx.x / G, lane = threadIdx.x % G;
  const int heads = a.heads[0] + a.heads[1];
  float* row = rows + sub * (a.d + 1);
  for (int h0 = blockIdx.y * per; h0 < heads; h0 += gridDim.y * per) {
    const int h = h0 + sub;
    const bool live = h < heads;
    const int w = live && h >= a.heads[0] ? 1 : 0;
    const int hh = h - (w ? a.heads[0] : 0);
    const T* x = reinterpret_cast<const T*>(a.x[w]) + r * a.stride[w] + (int64_t)hh * a.d;
    float v[NC][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = (c * G + lane) * 8;
      if (live && e < a.d) {
        load8<T>(x + e, v[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
      }
    }
    for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // correctly rounded square root and divide: the gain of every element
    const float rs = a.norm ? 1.0f / sqrtf(ss / (float)a.d + a.eps) : 1.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = (c * G + lane) * 8;
      if (live && e < a.d) {
        float g[8];
        if (a.norm && a.gain[w]) load8<float>(a.gain[w] + e, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[c][i] *= rs;
          if (a.norm && a.gain[w]) v[c][i] *= g[i];
          row[e + i] = v[c][i];
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = (c * G + lane) * 8;
      if (live && e < a.d) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = e + i - a.rope_off;
          if (j >= 0 && j < a.rope_dims) {
            const int p = a.half ? (j < half_dims ? j : j - half_dims) : j >> 1;
            const bool second = a.half ? j >= half_dims : (j & 1) != 0;
            const int step = a.half ? half_dims : 1;
            const float other = row[e + i + (second ? -step : step)];
            const float2 t = cs[p];
            v[c][i] = second ? fmaf(other, t.y, v[c][i] * t.x) : fmaf(v[c][i], t.x, -other * t.y);
          }
        }
        store8<T>(reinterpret_cast<T*>(a.out[w]) + r * a.out_stride[w] + (int64_t)hh * a.d + e, v[c]);
      }
    }
    __syncwarp();
  }
}

template <typename T>
csa_status launch_typed(const NormRopeArgs& a, int R, cudaStream_t st) {
  int G = 1;
  while (G < 32 && G * 8 < a.d) G <<= 1;
  const int per = kNrThreads / G, heads = a.heads[0] + a.heads[1];
  const int groups = (heads + per - 1) / per;
  // one CTA a token; few tokens: their heads spread over the SMs
  int gy = 1;
  while (gy < groups && (long long)R * gy < sm_count()) ++gy;
  const size_t smem = (size_t)(2 * (a.rope_dims / 2) + per * (a.d + 1)) * sizeof(float);
  csa_status st_ok = CSA_OK;
  auto kern = a.d > 256 ? qk_norm_rope_kernel<T, 2> : qk_norm_rope_kernel<T, 1>;
  if (smem > 48 * 1024 && !set_kernel_smem((const void*)kern, (int)smem)) return CSA_ERR_CUDA;
  CSA_LAUNCH(KK_NORM_ROPE, st,
             if (launch_maybe_pdl(true, kern, dim3((unsigned)R, (unsigned)gy), dim3(kNrThreads), smem,
                                  st, a, G) != cudaSuccess) st_ok = CSA_ERR_CUDA);
  return st_ok != CSA_OK ? st_ok : last_launch_status();
}

}  // namespace

csa_status launch_rope_freqs(const csa_rope& r, double* turns, cudaStream_t st) {
  const int n = r.rope_dims / 2;
  if (n == 0) return CSA_OK;
  CSA_LAUNCH(KK_ROPE_FREQS, st, rope_freqs_kernel<<<(n + 127) / 128, 128, 0, st>>>(r, turns));
  return last_launch_status();
}

csa_status launch_qk_norm_rope(const NormRopeArgs& a, int R, int act, cudaStream_t st) {
  return act == CSA_F32 ? launch_typed<float>(a, R, st) : launch_typed<__nv_bfloat16>(a, R, st);
}

}  // namespace csa
