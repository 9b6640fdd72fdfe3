// kv8_append.cu -- new tokens into the 8-bit KV cache (csa_kv8_append).
//
// A CTA owns one block of one KV head's K or V: it holds the block's new
// values in registers, forms max|x| over them, takes the least exponent e
// with max|x| <= 448 2^e (not below the one that the block's earlier slots
// already have) and stores code = E4M3(x 2^-e).  If e grew, the earlier codes
// are rescaled by a power of two, in place.
//
// What bounds it: for prompts the bytes; 32K tokens of 8 KV heads (d = 128, bf16)
// 37.9 us for 201 MB, 81% of the measured copy rate (K and V of all heads of a
// block of slots side by side in the grid: they lie together in the input).  For
// single tokens one chain of loads and a vote: 32 sequences 2.6 us in a graph.
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

// 8 values as loaded; the bits of their largest magnitude order as unsigned
// integers with infinities and NaN above every number
template <typename T> struct Chunk;
template <> struct Chunk<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 4 ? (i < 2 ? u.x : u.y) : (i < 6 ? u.z : u.w);
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  __device__ __forceinline__ uint32_t top() const {  // as fp32 bits
    const uint32_t m = 0x7fff7fffu;
    const uint32_t t = __vmaxu2(__vmaxu2(u.x & m, u.y & m), __vmaxu2(u.z & m, u.w & m));
    return max(t << 16, t & 0xffff0000u);
  }
};
template <> struct Chunk<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ float get(int i) const {
    const uint4& f = i < 4 ? a : b;
    return __uint_as_float((i & 3) == 0 ? f.x : (i & 3) == 1 ? f.y : (i & 3) == 2 ? f.z : f.w);
  }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fffffffu;
    return max(max(max(a.x & m, a.y & m), max(a.z & m, a.w & m)),
               max(max(b.x & m, b.y & m), max(b.z & m, b.w & m)));
  }
};

__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// largest value over the CTA; every thread gets it
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const uint32_t r = (threadIdx.x & 31) < kApThreads / 32 ? red[threadIdx.x & 31] : 0u;
  return __reduce_max_sync(0xffffffffu, r);
}

template <typename T, int D, int BLOCK>
__global__ void __launch_bounds__(kApThreads) kv8_append_kernel(AppendArgs a) {
  constexpr int RC = D / 8, chunks = BLOCK * RC;  // chunks of a slot, of the block
  constexpr int NC = (chunks + kApThreads - 1) / kApThreads;
  __shared__ uint32_t red[2][kApThreads / 32];
  pdl_wait();
  // K and V of all heads of a block of slots lie together in the input: side by side
  const int bt = blockIdx.x / (2 * a.H), wh = blockIdx.x % (2 * a.H), b = blockIdx.y;
  const int w = wh & 1, h = wh >> 1;
  const int old = a.n_old[b];
  int cnt = a.n_new ? a.n_new[b] : a.T;
  const bool first = bt == 0 && h == 0 && w == 0 && threadIdx.x == 0;
  if (first && (old < 0 || old > a.N || cnt < 0 || cnt > a.T || (long long)old + cnt > a.N))
    atomicOr(a.err, CSA_DEV_BAD_INDEX);
  if (old < 0 || old > a.N) return;
  cnt = min(max(cnt, 0), a.T);
  const int end = (int)min((long long)old + cnt, (long long)a.N);
  const int s0 = (old / BLOCK + bt) * BLOCK;  // first slot of this block
  const int lo = max(old, s0), hi = min(end, s0 + BLOCK);  // new slots [lo, hi)
  if (lo >= hi) return;
  // (selected, not indexed: an indexed argument is copied to local memory)
  const int64_t stride = w ? a.stride[1] : a.stride[0];
  uint8_t* exps = w ? a.exps[1] : a.exps[0];
  const T* x = reinterpret_cast<const T*>(w ? a.x[1] : a.x[0]) + ((int64_t)b * a.T + s0 - old) * stride +
               (int64_t)h * D;
  const int64_t blk = ((int64_t)b * a.H + h) * (a.N / BLOCK) + s0 / BLOCK;
  const int was = lo > s0 ? exps[blk] : 0;
  Chunk<T> v[NC];
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = c * kApThreads + threadIdx.x, s = i / RC;
    if (i < chunks && s >= lo - s0 && s < hi - s0) {
      v[c].load(x + s * stride + (i % RC) * 8);
      top = max(top, v[c].top());
    }
  }
  top = block_max(top, red[0]);
  const bool odd = top >= 0x7f800000u;  // an infinity or NaN among the values
  if (odd) {  // neither counts
    top = 0;
    bool nan = false;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = c * kApThreads + threadIdx.x, s = i / RC;
      if (i < chunks && s >= lo - s0 && s < hi - s0)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float f = fabsf(v[c].get(j));
          nan |= f != f;
          if (f < INFINITY) top = max(top, __float_as_uint(f));
        }
    }
    if (nan) atomicOr(a.err, CSA_DEV_NAN);
    top = block_max(top, red[1]);
  }
  int e = block_exponent(__uint_as_float(top));
  const int e_old = lo > s0 ? min(max(was - 127, kKv8MinExp), kKv8MaxExp) : e;
  e = max(e, e_old);
  const float f = pow2i(-e);  // e >= -110 and e <= 119: a normal number
  uint2* codes = reinterpret_cast<uint2*>((w ? a.codes[1] : a.codes[0]) + blk * (BLOCK * (int64_t)D));
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = c * kApThreads + threadIdx.x, s = i / RC;
    if (i >= chunks) continue;
    if (s >= lo - s0 && s < hi - s0) {
      float t[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = v[c].get(j) * f;
      if (odd)
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = t[j] == t[j] ? t[j] : 0.f;
      codes[i] = make_uint2(encode4(t[0], t[1], t[2], t[3]), encode4(t[4], t[5], t[6], t[7]));
    } else if (s < lo - s0 && e > e_old) {
      // earlier codes under the larger exponent: an exact shift of the
      // exponent, rounded again only where it ends among E4M3's subnormals
      const float g = e - e_old > 126 ? 0.f : pow2i(e_old - e);
      const uint2 u = codes[i];
      float t[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = e4m3_to_f32((uint8_t)((j < 4 ? u.x : u.y) >> (8 * (j & 3)))) * g;
      codes[i] = make_uint2(encode4(t[0], t[1], t[2], t[3]), encode4(t[4], t[5], t[6], t[7]));
    }
  }
  // (every thread read the old exponent before the barrier of block_max)
  if (threadIdx.x == 0) exps[blk] = (uint8_t)(e + 127);
}

template <typename T, int D>
auto pick(int block) {
  return block == 16 ? kv8_append_kernel<T, D, 16> : block == 32 ? kv8_append_kernel<T, D, 32>
         : block == 64 ? kv8_append_kernel<T, D, 64> : kv8_append_kernel<T, D, 128>;
}

template <typename T>
csa_status launch_typed(const AppendArgs& a, const csa_kv8_params& p, cudaStream_t st) {
  auto kern = p.d == 64 ? pick<T, 64>(p.block) : p.d == 128 ? pick<T, 128>(p.block) : pick<T, 256>(p.block);
  if ((long long)a.nbt * 2 * a.H > 0x7fffffffll || a.B > 65535) return CSA_ERR_SHAPE;
  csa_status ok = CSA_OK;
  CSA_LAUNCH(KK_KV8_APPEND, st,
             if (launch_maybe_pdl(true, kern, dim3((unsigned)(a.nbt * 2 * a.H), (unsigned)a.B), dim3(kApThreads), 0, st, a) !=
                 cudaSuccess) ok = CSA_ERR_CUDA);
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
