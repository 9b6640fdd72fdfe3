// kv8_attend.cuh -- what the two forms of csa_kv8_attend share: arguments, the
// line of units, conversions (kv8_attend.cu: few query rows a KV head;
// kv8_attend_tc.cu: many).
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kv8.h"
#include "sm100.cuh"

namespace csa {
namespace kv8 {

constexpr float kLog2e = 1.4426950408889634f;
// Tensor-core forms: 524 queries (7 heads a KV head, 2 of them, d = 128, bf16) over
// 1024 slots: one line 45 us, a CTA an item (8 units) 35; over 2048: 47.4 and 53.6.
constexpr int kTcJoinUnits = 8;
constexpr int kSms = 148;          // SMs that the choices below count with
constexpr int kMaxPlan = 1024;     // (sequence, row tile) pairs that the line of units holds
constexpr int kMaxGrid = 160;      // CTAs whose pieces the workspace holds (148 SMs)
// Value exponents within +-kTame: sums relative to the maximum of y neither
// overflow nor lose a term of weight.  Where a sequence has others (blocks of
// zeros, above all), its sum gets a maximum of its own, that of x.
constexpr int kTame = 40;
// The tensor cores cut off what they add to an accumulator, towards zero, and of
// products far below it all but a few bits.  bf16 prompts over values of one sign lost
// 1.3e-4 over 32K slots, 9e-4 over 128K and 8e-3 over 1M: after so many slots of an
// item O goes to a sum in memory and starts anew (256 queries over 1M slots, 64 heads, 8
// KV heads, d = 128: 8.80 -> 9.14 ms; 512 over 128K 2.18 -> 2.24).
constexpr int kPartSlots = 32768;

struct AttnArgs {
  const void* q;
  const int32_t* n_vis;
  const uint8_t* kc;
  const uint8_t* vc;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  const float* sink;
  void* out;
  float* blk_log;   // [B][H][Q G][NSB] log2 of each sub-block's weight sum (not normalised)
  float* row_log;   // [B][H][Q G] log2 of the row's denominator
  float* part_o;    // [grid][2][rows of a CTA][d] pieces of items that several CTAs share
  float4* sum_o;    // tensor-core forms, bf16, in parts: [grid][rows of a CTA][d] floats
  float4* part_ml;  // [grid][2][rows of a CTA] their M, reference of the sum, sum
  int* plan;        // [E + 1] units before each (sequence, row tile)
  float* acc;
  unsigned* err;
  int B, Q, H, G, N, NB, block;
  int sub, NSB;     // slots of a sub-block: min(block, 32); sub-blocks of N
  int shift, sub_shift;  // log2 of block and sub
  int RT, E, planned;
  int parts;        // O is summed up in parts (its CTAs may walk so many slots of an item)
  float scale2, decay;  // softmax scale times log2(e)
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int clamp_exp(int e) { return min(max(e, -126), 127); }

// four codes (a 32-bit word) -> two fp16 pairs
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// the last slot that queries of row tile rt see, plus one, over every `step`-th
// of them from `first` on; rows are query * G + head of the group, `rows` a tile
__device__ __forceinline__ int tile_max(const AttnArgs& a, int b, int rt, int rows, int first, int step) {
  const int j0 = (int)((int64_t)rt * rows / a.G);
  const int j1 = (int)min(((int64_t)rt * rows + rows - 1) / a.G, (int64_t)a.Q - 1);
  int n = 0;
#pragma unroll 4
  for (int j = j0 + first; j <= j1; j += step) {
    const int v = a.n_vis[(int64_t)b * a.Q + j];
    if (v > a.N) atomicOr(a.err, CSA_DEV_BAD_INDEX);
    n = max(n, min(v, a.N));
  }
  return n;
}

// CTA c of `grid` takes the units [cut(c), cut(c + 1)) of the line; grid is at
// most total, so every range holds a unit (the launch may have more CTAs)
__device__ __forceinline__ long long cut(long long c, long long total, int grid) {
  return c * total / grid;
}

// A walk along the line of units.
struct Cursor {
  int e, h, local, units, n;  // (sequence, row tile), KV head, unit in it, its units, n_max
  __device__ __forceinline__ void load(const int* before, const int* nmax) {
    units = before[e + 1] - before[e];
    n = nmax[e];
  }
  __device__ __forceinline__ void next(const int* before, const int* nmax, int H, int E) {
    if (++local < units) return;
    local = 0;
    if (++h < H) return;
    h = 0;
    do { ++e; } while (e < E && before[e + 1] == before[e]);
    if (e < E) load(before, nmax);
  }
};

// Where a CTA of THREADS threads begins: fills before / nmax (shared memory)
// and sets the cursor, the range [u0, u1) of the line and e_base ((sequence,
// row tile) of the line's first entry).  With a plan all units lie on one
// line, cut evenly over the CTAs; without, a CTA has one item.  False: the CTA
// has nothing to do.  All threads of the CTA call it.
template <int THREADS>
__device__ __forceinline__ bool begin_line(const AttnArgs& a, int rows, int unit, int* before, int* nmax,
                                           unsigned* scan_sh, Cursor& cur, long long& u0, long long& u1,
                                           int& e_base) {
  const int tid = threadIdx.x;
  e_base = 0;
  if (a.planned) {
    // so many lanes an entry that each has about four queries to look at
    int lpe = 1;
    while (lpe * 4 < rows / a.G + 1 && lpe < 32) lpe <<= 1;
    for (int first = 0; first < a.E; first += THREADS / lpe) {
      const int e = first + tid / lpe;
      int n = e < a.E ? tile_max(a, e / a.RT, e % a.RT, rows, tid % lpe, lpe) : 0;
      for (int o = lpe >> 1; o > 0; o >>= 1) n = max(n, __shfl_xor_sync(0xffffffffu, n, o));
      if (e < a.E && tid % lpe == 0) nmax[e] = n;
    }
    __syncthreads();
    const int per = (a.E + THREADS - 1) / THREADS;
    const int e0 = min(tid * per, a.E), e1 = min(e0 + per, a.E);
    unsigned mine = 0, all;
    for (int e = e0; e < e1; ++e) mine += (unsigned)((nmax[e] + unit - 1) / unit);
    unsigned at = block_exclusive_scan(mine, scan_sh, &all);
    for (int e = e0; e < e1; ++e) {
      before[e] = (int)at;
      at += (unsigned)((nmax[e] + unit - 1) / unit);
    }
    if (tid == 0) before[a.E] = (int)all;
    __syncthreads();
    if (blockIdx.x == 0)
      for (int e = tid; e <= a.E; e += THREADS) a.plan[e] = before[e];
    const long long total = (long long)all * a.H;
    const int grid = (int)min((long long)gridDim.x, total);
    if ((int)blockIdx.x >= grid) return false;
    u0 = cut(blockIdx.x, total, grid);
    u1 = cut(blockIdx.x + 1, total, grid);
    int lo = 0, hi = a.E;  // the last e with H * before[e] <= u0 that has units
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)before[mid] * a.H <= u0) lo = mid; else hi = mid;
    }
    cur.e = lo;
    cur.load(before, nmax);
    const int off = (int)(u0 - (long long)before[lo] * a.H);
    cur.h = off / cur.units;
    cur.local = off % cur.units;
  } else {
    const int e = (int)(blockIdx.x / a.H);
    if (tid < 32) {
      const int n = __reduce_max_sync(0xffffffffu, tile_max(a, e / a.RT, e % a.RT, rows, tid, 32));
      if (tid == 0) {
        before[0] = 0;
        before[1] = (n + unit - 1) / unit;
        nmax[0] = n;
      }
    }
    __syncthreads();
    e_base = e;
    cur.e = 0;
    cur.h = (int)(blockIdx.x % a.H);
    cur.local = 0;
    cur.load(before, nmax);
    u0 = 0;
    u1 = max(cur.units, 1);  // an item without slots still writes its zeros
  }
  return true;
}

// For an item [U0, U0 + units) of a line of `total` units: the CTAs that hold
// its first and last unit, and where a CTA put its piece (its first segment is
// piece 0, its last one piece 1).
struct Pieces {
  long long U0, total;
  int grid, c0, c1;
  __device__ __forceinline__ Pieces(const AttnArgs& a, int e, int h, int units, int launched) {
    total = (long long)a.plan[a.E] * a.H;
    grid = (int)min((long long)launched, total);
    U0 = (long long)a.plan[e] * a.H + (long long)h * units;
    // (clamped: a plan that another call overwrote, in a workspace that two of them share
    // against the rules, gives wrong pieces but no address outside of the workspace)
    c0 = (int)min(max(((U0 + 1) * grid - 1) / max(total, 1ll), 0ll), (long long)launched - 1);
    c1 = (int)min(max(((U0 + units) * grid - 1) / max(total, 1ll), (long long)c0), (long long)launched - 1);
  }
  __device__ __forceinline__ int64_t slot(int c) const {
    return (int64_t)c * 2 + (cut(c, total, grid) >= U0 ? 0 : 1);
  }
};

// Whether the units of all items go on one line: that evens the CTAs out, but the
// pieces then need a second kernel, which costs as much as `join` units.
inline bool on_a_line(long long items, int N, int unit, int sms, int join) {
  const long long per = (N + unit - 1) / unit;
  return (items + sms - 1) / sms * per > (items * per + sms - 1) / sms + join;
}
// and what the longest CTA then takes, in units
inline long long line_units(long long items, int N, int unit, int sms, int join) {
  const long long per = (N + unit - 1) / unit;
  return on_a_line(items, N, unit, sms, join) ? (items * per + sms - 1) / sms + join : (items + sms - 1) / sms * per;
}

}  // namespace kv8

// many query rows a KV head (kv8_attend_tc.cu: bf16, d <= 128; kv8_attend_tc1.cu):
// rows of a CTA
int kv8_attend_tc_rows();
int kv8_attend_tc1_rows();
csa_status launch_kv8_attend_tc1(const csa_kv8_params& p, kv8::AttnArgs& a, cudaStream_t st);
csa_status launch_kv8_attend_tc(const csa_kv8_params& p, kv8::AttnArgs& a, cudaStream_t st);

}  // namespace csa
