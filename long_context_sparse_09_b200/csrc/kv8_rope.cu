// kv8_rope.cu -- per-head RMSNorm and rotation of queries and keys in one
// pass (csa_qk_norm_rope), and the table of angles it reads.
//
//   y = x * gain / sqrt(mean(x^2) + eps);  (a, b) -> (a cos - b sin, a sin + b cos)
//
// A CTA owns a few tokens: it forms their cos / sin once (fp64 turns, reduced to
// a fraction of a turn before fp32) and walks their heads, a group of lanes a
// head, 8 elements a lane and chunk.  Where a pair's elements are in one lane's
// chunk, or in the same place of two lanes' chunks, they meet in registers;
// elsewhere the row goes through shared memory.
//
// What bounds it: for prompts the bytes, each read and written once; 32K tokens
// of 64 + 8 heads (d = 128, bf16, 64 rotated dims) 208 to 216 us for 1.21 GB, by
// machine, 85 to 88% of the measured copy rate.  For few tokens the chain position -> angles -> heads: four
// tokens of 64 + 8 heads 3.0 us in a graph.
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

// 8 values as loaded
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 4 ? (i < 2 ? u.x : u.y) : (i < 6 ? u.z : u.w);
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ float get(int i) const {
    const float4& f = i < 4 ? a : b;
    return (i & 3) == 0 ? f.x : (i & 3) == 1 ? f.y : (i & 3) == 2 ? f.z : f.w;
  }
};
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// How a pair's elements meet: both in a lane's chunk (interleaved, even
// offset), in chunks of two lanes of the head's group (halves of whole chunks,
// d <= 256), or anywhere (through shared memory).
enum PairMode { kInChunk = 0, kAcrossLanes = 1, kThroughSmem = 2 };

// G lanes a head (a power of two, at least d / 8 up to 32), NC chunks a lane
// (2 only for d > 256).  A CTA takes `tokens` tokens; a group stays with one
// of them and walks its heads, so gain times cosine and sine of the lane's
// elements, the same in every head, stay in registers:
//   out = rs (v A + partner B).
template <typename T, int MODE, int NC, int G>
__global__ void __launch_bounds__(kNrThreads, MODE == kThroughSmem ? 2 : sizeof(T) == 4 ? 3 : 4)
qk_norm_rope_kernel(NormRopeArgs a, int R, int tokens, int q_ctas) {
  extern __shared__ float sm[];
  float2* cs = reinterpret_cast<float2*>(sm);                     // [tokens][rope_dims / 2]
  float* rows = sm + 2 * (a.rope_dims / 2) * tokens;              // [threads / G][d + 1], kThroughSmem
  // heads of a group whose loads are in flight together
  constexpr int U = MODE == kThroughSmem ? 1 : sizeof(T) == 4 ? 2 : 3;
  pdl_wait();
  const int half_dims = a.rope_dims / 2;
  const int sub = threadIdx.x / G, lane = threadIdx.x % G;
  const int groups = kNrThreads / G / tokens;                     // of a token
  const int tok = sub / groups;
  const int64_t r = (int64_t)blockIdx.x * tokens + tok;
  // q_ctas > 0: that many CTAs of a token for its queries, the others for its keys
  const bool keys = q_ctas > 0 && (int)blockIdx.y >= q_ctas;
  const int y = blockIdx.y - (keys ? q_ctas : 0);
  const int h_first = y * groups;
  const int first = h_first + sub % groups;
  const int step = (q_ctas == 0 ? 1 : keys ? gridDim.y - q_ctas : q_ctas) * groups;
  const int jump = step * a.d;
  const int w0 = keys ? 1 : 0, w1 = q_ctas > 0 && !keys ? 1 : 2;
  const float inv_d = 1.f / (float)a.d;
  Raw8<T> raw[U][NC];
  const T* src = reinterpret_cast<const T*>(a.x[w0]) + r * a.stride[w0] + (int64_t)first * a.d + lane * 8;
  auto fetch = [&](int h, int n) {
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (r < R && h + k * step < n && (c * G + lane) * 8 < a.d) raw[k][c].load(src + k * jump + c * G * 8);
  };
  fetch(first, a.heads[w0]);  // the first heads arrive while the angles are formed
  auto gains = [&](int w, int e, float (&g)[8]) {  // of the 8 elements from e on
    const float* gain = a.norm ? a.gain[w] : nullptr;
    if (gain && e < a.d) {
      const float4 x = *reinterpret_cast<const float4*>(gain + e);
      const float4 y = *reinterpret_cast<const float4*>(gain + e + 4);
      g[0] = x.x; g[1] = x.y; g[2] = x.z; g[3] = x.w;
      g[4] = y.x; g[5] = y.y; g[6] = y.z; g[7] = y.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = 1.f;
    }
  };
  float A[NC][8], B[8];
  bool turned[4] = {false, false, false, false};  // by pair (kInChunk), or all alike
  const int j0 = lane * 8 - a.rope_off;           // of the lane's chunk among the rotated dims
  const bool second = MODE == kAcrossLanes && j0 >= half_dims;
  const int other = second ? -half_dims : half_dims;
  int from = threadIdx.x & 31;
  if (MODE == kAcrossLanes) {
    turned[0] = j0 >= 0 && j0 < a.rope_dims;
    if (turned[0]) from += other / 8;
  }
  auto all_gains = [&](int w) {
#pragma unroll
    for (int c = 0; c < NC; ++c) gains(w, (c * G + lane) * 8, A[c]);
    if (MODE == kAcrossLanes && turned[0]) gains(w, lane * 8 + other, B);
  };
  all_gains(w0);
  for (int i = threadIdx.x; i < half_dims * tokens; i += kNrThreads) {
    const int64_t row = (int64_t)blockIdx.x * tokens + i / half_dims;
    if (row >= R) break;
    const double t = (double)a.pos[row] * a.turns[i % half_dims];
    const float f = (float)(2.0 * (t - rint(t)));   // half turns in [-1, 1]
    float s, c;
    sincospif(f, &s, &c);
    cs[i] = make_float2(c * a.mscale, s * a.mscale);
  }
  __syncthreads();
  cs += tok * half_dims;
  float* row = rows + sub * (a.d + 1);
#pragma unroll 1
  for (int w = w0; w < w1; ++w) {  // queries, then keys
    const int n = a.heads[w];
    if (n == 0) break;
    T* dst = reinterpret_cast<T*>(a.out[w]) + r * a.out_stride[w] + (int64_t)first * a.d + lane * 8;
    if (w > w0) {
      src = reinterpret_cast<const T*>(a.x[1]) + r * a.stride[1] + (int64_t)first * a.d + lane * 8;
      fetch(first, n);
      all_gains(w);
    }
    // factors of this lane's elements
    if constexpr (MODE == kInChunk) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int j = j0 + 2 * p;
        turned[p] = j >= 0 && j < a.rope_dims;
        const float2 t = turned[p] ? cs[j >> 1] : make_float2(1.f, 0.f);
        B[2 * p] = -A[0][2 * p + 1] * t.y;
        B[2 * p + 1] = A[0][2 * p] * t.y;
        A[0][2 * p] *= t.x;
        A[0][2 * p + 1] *= t.x;
      }
    } else if constexpr (MODE == kAcrossLanes) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 t = turned[0] ? cs[j0 + i - (second ? half_dims : 0)] : make_float2(1.f, 0.f);
        A[0][i] *= t.x;
        B[i] = turned[0] ? B[i] * (second ? t.y : -t.y) : 0.f;
      }
    }
#pragma unroll 1
    for (int h0 = 0; h_first + h0 < n; h0 += U * step) {  // (all lanes of the CTA together)
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const bool live = r < R && first + h0 + k * step < n;
        float v[NC][8];
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const bool have = live && (c * G + lane) * 8 < a.d;
          float part = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[c][i] = raw[k][c].get(i);
            part = fmaf(v[c][i], v[c][i], part);
          }
          ss += have ? part : 0.f;  // (what was not loaded does not count)
        }
        float rs = 1.f;
        if (a.norm) {
#pragma unroll
          for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          rs = rsqrtf(fmaf(ss, inv_d, a.eps));
        }
        float y[NC][8];
        if constexpr (MODE == kInChunk) {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const float x0 = v[0][2 * p], x1 = v[0][2 * p + 1];
            y[0][2 * p] = fmaf(x0, A[0][2 * p], (turned[p] ? x1 : 0.f) * B[2 * p]) * rs;
            y[0][2 * p + 1] = fmaf(x1, A[0][2 * p + 1], (turned[p] ? x0 : 0.f) * B[2 * p + 1]) * rs;
          }
        } else if constexpr (MODE == kAcrossLanes) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = __shfl_sync(0xffffffffu, v[0][i], from);
            y[0][i] = fmaf(v[0][i], A[0][i], (turned[0] ? x : 0.f) * B[i]) * rs;
          }
        } else {
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              y[c][i] = v[c][i] * (rs * A[c][i]);
              if ((c * G + lane) * 8 < a.d) row[(c * G + lane) * 8 + i] = y[c][i];
            }
          __syncwarp();
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int e = (c * G + lane) * 8 + i, j = e - a.rope_off;
              if (e >= a.d || j < 0 || j >= a.rope_dims) continue;
              const int p = a.half ? (j < half_dims ? j : j - half_dims) : j >> 1;
              const bool second = a.half ? j >= half_dims : (j & 1) != 0;
              const int off = a.half ? half_dims : 1;
              const float x = row[e + (second ? -off : off)];
              const float2 t = cs[p];
              y[c][i] = second ? fmaf(x, t.y, y[c][i] * t.x) : fmaf(y[c][i], t.x, -x * t.y);
            }
          __syncwarp();
        }
        if (live)
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if ((c * G + lane) * 8 < a.d) store8(dst + k * jump + c * G * 8, y[c]);
      }
      src += (int64_t)U * jump;
      dst += (int64_t)U * jump;
      fetch(first + h0 + U * step, n);
    }
  }
}

template <typename T, int MODE, int NC, int G>
csa_status launch_group(const NormRopeArgs& a, int R, cudaStream_t st) {
  constexpr int per = kNrThreads / G;
  // four or eight tokens a CTA where that still gives every SM work (a group's
  // factors then serve so many more heads; 32K tokens of 64 + 8 heads: 222 and 208
  // us, 1,500 of 32 + 8: 12.7 and 14.7); few tokens: one a CTA, and with fewer tokens
  // than SMs their heads spread over several
  int tokens = R >= 16 * sm_count() ? 8 : R >= 4 * sm_count() ? 4 : 1;
  // more of them where the heads leave groups idle and there are CTAs enough
  while (tokens >= 4 && 2 * tokens <= per && per / (2 * tokens) >= a.heads[0] && R >= 8 * tokens * sm_count()) tokens *= 2;
  const bool spread = R < sm_count();
  const int q_ctas = spread ? (a.heads[0] + per - 1) / per : 0;
  const int gy = spread ? q_ctas + (a.heads[1] + per - 1) / per : 1;
  const size_t smem = (size_t)(2 * (a.rope_dims / 2) * tokens + (MODE == kThroughSmem ? per * (a.d + 1) : 0)) * sizeof(float);
  auto kern = qk_norm_rope_kernel<T, MODE, NC, G>;
  if (smem > 48 * 1024 && !set_kernel_smem((const void*)kern, (int)smem)) return CSA_ERR_CUDA;
  csa_status ok = CSA_OK;
  CSA_LAUNCH(KK_NORM_ROPE, st,
             if (launch_maybe_pdl(true, kern, dim3((unsigned)((R + tokens - 1) / tokens), (unsigned)gy),
                                  dim3(kNrThreads), smem, st, a, R, tokens, q_ctas) != cudaSuccess)
               ok = CSA_ERR_CUDA);
  return ok != CSA_OK ? ok : last_launch_status();
}

template <typename T, int MODE>
csa_status launch_mode(const NormRopeArgs& a, int R, cudaStream_t st) {
  if (a.d <= 64) return launch_group<T, MODE, 1, 8>(a, R, st);
  if (a.d <= 128) return launch_group<T, MODE, 1, 16>(a, R, st);
  return launch_group<T, MODE, 1, 32>(a, R, st);
}

template <typename T>
csa_status launch_typed(const NormRopeArgs& a, int R, cudaStream_t st) {
  if (a.d > 256) return launch_group<T, kThroughSmem, 2, 32>(a, R, st);
  if (a.rope_dims == 0 || (!a.half && a.rope_off % 2 == 0)) return launch_mode<T, kInChunk>(a, R, st);
  if (a.half && a.rope_off % 8 == 0 && a.rope_dims % 16 == 0) return launch_mode<T, kAcrossLanes>(a, R, st);
  return launch_mode<T, kThroughSmem>(a, R, st);
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
