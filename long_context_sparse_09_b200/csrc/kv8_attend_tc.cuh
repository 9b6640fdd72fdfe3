// kv8_attend_tc.cuh -- what the two tensor-core kernels of csa_kv8_attend share
// (kv8_attend_tc.cu: two streams of 128 query rows; kv8_attend_tc1.cu: 128 rows,
// for fp32 activations and d = 256).
#pragma once

#include "kv8_attend.cuh"

namespace csa {
namespace kv8 {

using namespace sm100;

// The maximum may lag by 2^8, so that few tiles rescale O (a 32-row warp does it
// together): p = 2^(y - M + 7) stays below fp16's 2^16 and keeps 11 bits down
// to 2^-21 of 2^M.
constexpr float kTcLazy = 8.f, kTcShift = 7.f;
constexpr int kTcThreads = 416;  // 2 softmax warpgroups, 1 that widens, the MMA warp
constexpr int kTcJoinRows = 16;  // rows of a join CTA
// Loads and stores of tensor memory are the whole warp's (.sync.aligned), and rows
// differ in what they store and see: wherever a branch on the row lies between two of
// them, a __syncwarp() brings the lanes together again.

// 16 bytes of codes (not kept in L1), or zeros
__device__ __forceinline__ uint4 ld_stream_if(bool yes, const uint8_t* p) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "mov.u32 %3, 0;\n\t@q ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((int)yes));
  return v;
}

// two products and sums, two sums an instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// 2^z of a pair, z in [-inf, 127): z = n + r with n the nearest integer (Cody and
// Waite's reduction), 2^r a minimax polynomial of degree 4 on [-1/2, 1/2] that is 1 at
// 0 (relative error 2.9e-6, a hundredth of p's rounding to fp16), n added to the
// exponent.  z from -127 down, masked slots among it: n = -127, r = 0, which adds up
// to the bits of 0.  A quarter of the exponentials go this way, beside the special
// function unit (2.33 -> 2.21 ms at the size above; a half: 2.32)
__device__ __forceinline__ float2 exp2_poly(float2 z) {
  const float2 big = make_float2(12582912.f, 12582912.f), neg = make_float2(-12582912.f, -12582912.f);
  z.x = fmaxf(z.x, -127.f);
  z.y = fmaxf(z.y, -127.f);
  const float2 t = add2(z, big), n = add2(t, neg);
  const float2 r = fma2(n, make_float2(-1.f, -1.f), z);
  float2 p = fma2(r, make_float2(0.009585382f, 0.009585382f), make_float2(0.055906627f, 0.055906627f));
  p = fma2(p, r, make_float2(0.24024038f, 0.24024038f));
  p = fma2(p, r, make_float2(0.6931242f, 0.6931242f));
  p = fma2(p, r, make_float2(1.f, 1.f));
  return make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23)),
                     __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23)));
}


// The warpgroup that widens (threads 256-383 of the CTA): the codes of the units
// [u0, u1) from the cursor on as fp16 into a ring of NS tiles of KT slots, K and V
// in turn.  A tile is [D / 64][KT][64] fp16 in the 128-byte swizzle layout: the
// K-major operand of Q K^T and the MN-major one of P V.  Slots that no query of
// the item sees become zeros.
template <int D, int KT, int NS>
__device__ __forceinline__ void widen_role(const AttnArgs& a, Cursor pre, long long u0, long long u1, int e_base,
                                           const int* before, const int* nmax, uint8_t* ring, uint64_t* kv_full,
                                           uint64_t* kv_empty, volatile int* abort_sm) {
  constexpr int CH = D / 16;                         // 16-byte chunks of a slot
  constexpr int PER = 128 / CH;                      // slots a pass
  constexpr int NP = KT / PER;                       // passes
  // (every other four chunks of a row go to the neighbouring row's lanes: the
  // blocks of 64 dims lie on the same banks, the rows of a pair on different ones)
  const int t = threadIdx.x - 256, c = t % CH, first = t / CH ^ ((c >> 2) & 1), lane = threadIdx.x & 31;
  // a tile's registers are loaded again as soon as it is in the ring
  int64_t from = 0;  // of this thread's chunk of the next tile's first slot
  int left = 0;      // slots of that tile that a query sees
  auto locate = [&]() {
    // (from memory to L2 three units ahead: the loads a unit ahead cover L2 only;
    // 2,488 -> 2,427 us for 2048 queries over 32K slots that are not in L2)
    const int ahead = min(pre.n - (pre.local + 3) * KT, KT) * D;
    if (t == 0 && ahead > 0) {
      const int64_t at = (((int64_t)((pre.e + e_base) / a.RT) * a.H + pre.h) * a.N + (int64_t)(pre.local + 3) * KT) * D;
      bulk_prefetch_l2(a.kc + at, ahead);
      bulk_prefetch_l2(a.vc + at, ahead);
    }
    from = (((int64_t)((pre.e + e_base) / a.RT) * a.H + pre.h) * a.N + (int64_t)pre.local * KT + first) * D + c * 16;
    left = pre.n - pre.local * KT - first;
  };
  auto fetch = [&](uint4 (&r)[NP], const uint8_t* codes) {
#pragma unroll
    for (int p = 0; p < NP; ++p) r[p] = ld_stream_if(p * PER < left, codes + from + p * PER * D);
  };
  int at = 0;  // tiles written to the ring
  auto put = [&](const uint4 (&r)[NP]) -> bool {
    const int s = at % NS;
    if (!__all_sync(0xffffffffu, mbar_wait(&kv_empty[s], ((at / NS) & 1) ^ 1, abort_sm))) return false;
    uint8_t* dst = ring + s * (KT * D * 2) + (c >> 2) * (KT * 128);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int slot = p * PER + first;
      uint4 w[2];
      widen4(r[p].x, w[0].x, w[0].y);
      widen4(r[p].y, w[0].z, w[0].w);
      widen4(r[p].z, w[1].x, w[1].y);
      widen4(r[p].w, w[1].z, w[1].w);
      uint8_t* line = dst + slot * 128;
      const int c0 = 2 * (c & 3);
      *reinterpret_cast<uint4*>(line + ((c0 ^ (slot & 7)) << 4)) = w[0];
      *reinterpret_cast<uint4*>(line + (((c0 + 1) ^ (slot & 7)) << 4)) = w[1];
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&kv_full[s]);
    ++at;
    return true;
  };
  if (pre.units == 0) return;
  long long up = u0;   // unit whose tiles are fetched next
  auto step = [&]() {  // to the next unit; none: nothing is loaded
    if (++up < u1) {
      pre.next(before, nmax, a.H, a.E);
      locate();
    } else {
      left = 0;
    }
  };
  uint4 k0[NP], v0[NP];
  locate();
  fetch(k0, a.kc);
  fetch(v0, a.vc);
  step();
  for (long long u = u0; u < u1; ++u) {
    if (!put(k0)) return;
    fetch(k0, a.kc);
    if (!put(v0)) return;
    fetch(v0, a.vc);
    step();
  }
}

// Joins the pieces of the items that several CTAs share, a warp two rows at a
// time; rows of sequences without slots get their zeros here.
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(256) kv8_join(AttnArgs a, int launched) {
  pdl_wait();
  constexpr int parts = ROWS / kTcJoinRows, U = kTcJoinRows / 8;
  const int64_t item = blockIdx.x / parts;
  const int e = (int)(item / a.H), h = (int)(item % a.H), b = e / a.RT, rt = e % a.RT;
  const int units = a.plan[e + 1] - a.plan[e], lane = threadIdx.x & 31;
  const int r0 = (int)(blockIdx.x % parts) * kTcJoinRows + (threadIdx.x >> 5) * U;
  float v[U][D / 32];
#pragma unroll
  for (int k = 0; k < U; ++k)
#pragma unroll
    for (int i = 0; i < D / 32; ++i) v[k][i] = 0.f;
  if (units > 0) {
    const Pieces pc(a, e, h, units, launched);
    if (pc.c0 == pc.c1) return;
    float M[U], MX[U], L[U];
#pragma unroll
    for (int k = 0; k < U; ++k) M[k] = MX[k] = -INFINITY, L[k] = 0.f;
#pragma unroll 2
    for (int c = pc.c0; c <= pc.c1; ++c) {
      const float4* p = a.part_ml + pc.slot(c) * ROWS + r0;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        M[k] = fmaxf(M[k], p[k].x);
        MX[k] = fmaxf(MX[k], p[k].y);
      }
    }
#pragma unroll 2
    for (int c = pc.c0; c <= pc.c1; ++c) {
      const int64_t sl = pc.slot(c) * ROWS + r0;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float4 p = a.part_ml[sl + k];
        const float f = p.x == -INFINITY ? 0.f : fast_exp2(p.x - M[k]);
        L[k] = fmaf(p.z, p.y == -INFINITY ? 0.f : fast_exp2(p.y - MX[k]), L[k]);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) v[k][i] = fmaf(a.part_o[(sl + k) * D + i * 32 + lane], f, v[k][i]);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t rho = (int64_t)rt * ROWS + r0 + k;
      if (rho >= (int64_t)a.Q * a.G) break;
      const int j = (int)(rho / a.G);
      if (a.sink) L[k] += fast_exp2(a.sink[h * a.G + (int)(rho % a.G)] * kLog2e - MX[k]);
      if (a.row_log && lane == 0) a.row_log[((int64_t)b * a.H + h) * a.Q * a.G + rho] = log2f(L[k]) + MX[k];
      const bool sees = a.n_vis[(int64_t)b * a.Q + j] > 0;
      const float inv = 0x1p-7f / L[k], gap = fast_exp2(M[k] - MX[k]);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) v[k][i] = sees ? v[k][i] * inv * gap : 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int64_t rho = (int64_t)rt * ROWS + r0 + k;
    if (rho >= (int64_t)a.Q * a.G) return;
    T* out = reinterpret_cast<T*>(a.out) +
                         (((int64_t)b * a.Q + rho / a.G) * a.H * a.G + h * a.G + rho % a.G) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) out[i * 32 + lane] = from_f32<T>(v[k][i]);
  }
}

}  // namespace kv8
}  // namespace csa
