// kv8_append.cu -- new tokens into the 8-bit KV cache (csa_kv8_append).
//
// A CTA owns one block of one KV head's K or V: it holds the block's new
// values in registers, forms max|x| over them, takes the least exponent e
// with max|x| <= 448 2^e (not below the one that the block's earlier slots
// already have) and stores code = E4M3(x 2^-e).  If e grew, the earlier codes
// are rescaled by a power of two, in place.
#include "common.cuh"
#include "kv8.h"

namespace csa {

namespace {

constexpr int kApThreads = 256;

struct AppendArgs {
  const void* x[2];
  int64_t stride[2];
  uint8_t* codes[2];
  uint8_t* exps[2];
  const int32_t* n_old;
  const int32_t* n_new;
  unsigned* err;
  int B, T, H, N, nbt;  // nbt: blocks a sequence can touch
};

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// least e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), within the cache's range
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int ex = (int)(u >> 23) - 127;  // amax is finite, not negative; subnormal: -127
  const int e = ex - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kKv8MinExp), kKv8MaxExp);
}

template <typename T> struct Chunk;  // 8 values as loaded
template <> struct Chunk<__nv_bfloat16> {
  uint4 u;
  __device__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ float get(int i) const {
    const uint32_t w = i < 4 ? (i < 2 ? u.x : u.y) : (i < 6 ? u.z : u.w);
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
};
template <> struct Chunk<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ float get(int i) const {
    const float4& f = i < 4 ? a : b;
    return (i & 3) == 0 ? f.x : (i & 3) == 1 ? f.y : (i & 3) == 2 ? f.z : f.w;
  }
};

// codes of four scaled values (NaN: 0)
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  a = a == a ? a : 0.f; b = b == b ? b : 0.f;
  c = c == c ? c : 0.f; d = d == d ? d : 0.f;
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// NC chunks of 8 values a thread: block * d / 8 chunks over the CTA
template <typename T, int NC>
__global__ void __launch_bounds__(kApThreads) kv8_append_kernel(AppendArgs a, int d, int block) {
  __shared__ float red[32];
  pdl_wait();
  int64_t id = blockIdx.x;
  const int w = (int)(id & 1);
  id >>= 1;
  const int h = (int)(id % a.H);
  id /= a.H;
  const int bt = (int)(id % a.nbt), b = (int)(id / a.nbt);
  const int old = a.n_old[b];
  int cnt = a.n_new ? a.n_new[b] : a.T;
  const bool first = bt == 0 && h == 0 && w == 0 && threadIdx.x == 0;
  if (first && (old < 0 || old > a.N || cnt < 0 || cnt > a.T ||
                (long long)old + cnt > a.N))
    atomicOr(a.err, CSA_DEV_BAD_INDEX);
  if (old < 0 || old > a.N) return;
  cnt = min(max(cnt, 0), a.T);
  const int end = (int)min((long long)old + cnt, (long long)a.N);
  const int s0 = (old / block + bt) * block;  // first slot of this block
  if (s0 >= end) return;
  const int lo = max(old, s0), hi = min(end, s0 + block);  // new slots [lo, hi)
  const int row_chunks = d / 8, chunks = block * row_chunks;
  const T* x = reinterpret_cast<const T*>(a.x[w]) + (int64_t)b * a.T * a.stride[w] + (int64_t)h * d;
  Chunk<T> v[NC];
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = c * kApThreads + threadIdx.x;
    const int s = s0 + i / row_chunks;
    if (i < chunks && s >= lo && s < hi) {
      v[c].load(x + (int64_t)(s - old) * a.stride[w] + (i % row_chunks) * 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = fabsf(v[c].get(j));
        nan |= f != f;
        amax = fmaxf(amax, f < INFINITY ? f : 0.f);  // NaN and infinities do not count
      }
    }
  }
  if (nan) atomicOr(a.err, CSA_DEV_NAN);
  amax = block_reduce<true>(amax, red);
  const int64_t blk = ((int64_t)b * a.H + h) * (a.N / block) + s0 / block;
  int e = block_exponent(amax);
  const int e_old = lo > s0 ? min(max((int)a.exps[w][blk] - 127, kKv8MinExp), kKv8MaxExp) : e;
  e = max(e, e_old);
  const float f = pow2i(-e);  // e >= -110 and e <= 119: a normal number
  uint8_t* codes = a.codes[w] + blk * block * (int64_t)d;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = c * kApThreads + threadIdx.x;
    const int s = s0 + i / row_chunks;
    if (i >= chunks) continue;
    if (s >= lo && s < hi) {
      uint2 o;
      o.x = encode4(v[c].get(0) * f, v[c].get(1) * f, v[c].get(2) * f, v[c].get(3) * f);
      o.y = encode4(v[c].get(4) * f, v[c].get(5) * f, v[c].get(6) * f, v[c].get(7) * f);
      reinterpret_cast<uint2*>(codes)[i] = o;
    } else if (s < lo && e > e_old) {
      // earlier codes under the larger exponent: an exact shift of the
      // exponent, rounded again only where it ends among E4M3's subnormals
      const float g = e - e_old > 126 ? 0.f : pow2i(e_old - e);
      const uint2 u = reinterpret_cast<const uint2*>(codes)[i];
      float t[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = e4m3_to_f32((uint8_t)((j < 4 ? u.x : u.y) >> (8 * (j & 3)))) * g;
      uint2 o;
      o.x = encode4(t[0], t[1], t[2], t[3]);
      o.y = encode4(t[4], t[5], t[6], t[7]);
      reinterpret_cast<uint2*>(codes)[i] = o;
    }
  }
  __syncthreads();  // every thread has read the old exponent
  if (threadIdx.x == 0) a.exps[w][blk] = (uint8_t)(e + 127);
}

template <typename T>
csa_status launch_typed(const AppendArgs& a, const csa_kv8_params& p, cudaStream_t st) {
  const int chunks = p.block * p.d / 8, per = (chunks + kApThreads - 1) / kApThreads;
  auto kern = per <= 1 ? kv8_append_kernel<T, 1>
              : per <= 2 ? kv8_append_kernel<T, 2>
              : per <= 4 ? kv8_append_kernel<T, 4>
              : per <= 8 ? kv8_append_kernel<T, 8> : kv8_append_kernel<T, 16>;
  const long long ctas = 2ll * a.H * a.nbt * a.B;
  if (ctas > 0x7fffffffll) return CSA_ERR_SHAPE;
  csa_status ok = CSA_OK;
  CSA_LAUNCH(KK_KV8_APPEND, st,
             if (launch_maybe_pdl(true, kern, dim3((unsigned)ctas), dim3(kApThreads), 0, st, a, p.d,
                                  p.block) != cudaSuccess) ok = CSA_ERR_CUDA);
  return ok != CSA_OK ? ok : last_launch_status();
}

}  // namespace

csa_status launch_kv8_append(const csa_kv8_params& p, int B, int T, const void* k,
                             int64_t k_stride, const void* v, int64_t v_stride,
                             const int32_t* n_old, const int32_t* n_new, const Kv8Cache& c,
                             cudaStream_t st) {
  AppendArgs a;
  a.x[0] = k; a.x[1] = v;
  a.stride[0] = k_stride; a.stride[1] = v_stride;
  a.codes[0] = c.kc; a.codes[1] = c.vc;
  a.exps[0] = c.k_exp; a.exps[1] = c.v_exp;
  a.n_old = n_old;
  a.n_new = n_new;
  a.err = device_error_word();
  if (a.err == nullptr) return CSA_ERR_CUDA;
  a.B = B; a.T = T; a.H = p.n_kv; a.N = p.N;
  // T tokens from the last slot of a block on touch this many blocks at most
  a.nbt = (int)(((long long)T + p.block - 2) / p.block) + 1;
  if (a.nbt > p.N / p.block) a.nbt = p.N / p.block;
  return p.act == CSA_F32 ? launch_typed<float>(a, p, st) : launch_typed<__nv_bfloat16>(a, p, st);
}

}  // namespace csa
