// kv8_attend_tc.cu -- attention over the 8-bit KV cache for many query rows a
// KV head (prompt chunks), on the 5th-generation tensor cores.
//
// The mathematics is that of kv8_attend.cu: with x = scale log2(e) q . k and
// y = x + ve, out = sum 2^(y - M) c / sum 2^(y - ve - M), both products over
// codes widened to fp16 (exact), every power of two in an exponent.
//
// A CTA owns 256 query rows of a KV head (rows are query * G + head of the
// group) as two streams of 128, and walks the slots in tiles of 128:
//   S_s = Q_s K^T      tcgen05.mma, both operands in shared memory
//   P_s = 2^(y - M + 7) by stream s's warpgroup, a thread a row: S is read
//         from TMEM for its maximum and again, 32 slots at a time, for P, which
//         goes back as fp16 over the front half of S (all of S in registers
//         spills: 2.9 ms instead of 2.2 at the size below)
//   O_s += P_s V       tcgen05.mma, P from TMEM, V MN-major in shared memory
// While a stream's softmax runs, the tensor cores can work for the other one.  A
// third warpgroup widens the codes: 16-byte global loads (a tile ahead, in
// registers) -> fp16 in the 128-byte swizzle layout, K and V tiles alternating
// in one ring.  All tiles of the call lie on one line, cut evenly over the SMs;
// the pieces of items that several CTAs share are joined by kv8_join.
//
// What bounds it: the latency of a stream's chain S -> maximum -> P -> P V.  A pair of
// tiles (both streams) takes 4,700 cycles; its products take 2,060 of the tensor cores,
// the two softmax warps of a scheduler 2,015 for exponentials, sums and packing
// (measured without products; 1,536 of them the special function unit's) and 470 for
// the maxima, and they overlap only in part: no pipe is busy half of the time.
// Without P the kernel takes 1.37 ms, with half of it 1.50.  2048 queries of 64 heads
// over 32K slots of 8 KV heads (d = 128):
// 2.17 ms, 980 TFLOP/s, 61% of the measured bf16 rate (2.39 to 2.42 in long runs, under
// the power limit); on mma.sync (kv8_attend.cu) 11.4 ms.  Tiles of 64 slots with two S
// buffers a stream took 2.49 ms (a product with N = 64 costs as much as one with N =
// 128), the products issued by the softmax warps themselves 2.6 ms, four softmax
// warpgroups of half a tile each 2.94.
#include "kv8_attend_tc.cuh"

namespace csa {

using namespace kv8;

namespace {

constexpr int kTcRows = 256;     // query rows of a CTA: two streams of 128
constexpr int kTcTile = 128;     // slots of a tile

template <int D>
struct Tc {
  static constexpr int row_tile = kTcTile * D * 2;   // 128 rows of fp16: a stream's Q, a K or V tile
  static constexpr int NS = D == 64 ? 8 : 4;         // K and V tiles in the ring
  static constexpr int q = 0;
  static constexpr int ring = 2 * row_tile;
  static constexpr int table = ring + NS * row_tile;           // [8 warps][2][32] float4
  static constexpr int plan = table + 8 * 2 * 32 * 16;         // units before, n_max: [E + 1], [E]
  static constexpr int bars = plan + (2 * kMaxPlan + 2) * 4;
  static constexpr int mem_ref = bars + (2 * NS + 8) * 8 + 16;  // [256] M of the rows' sums in memory
  static constexpr int total = mem_ref + kTcRows * 4;
  static_assert(total + 1024 <= 232448, "shared memory");
};

// O of a row goes to its sum in memory: sum = f sum (nothing: `begin`) + O.  (Not inline:
// registers of the loop around it would be spilled.)
template <int D>
__device__ __noinline__ void put_part(uint32_t tO, float4* sum, float f, bool begin) {
  __syncwarp();
  tmem_wait_st();  // O may just have been rescaled
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    float w[16];
    tmem_ld16(tO + c, w);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; k += 4) {
      float4* at = sum + (c + k) / 4 * kTcRows;
      const float4 o = begin ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldcg(at);
      *at = make_float4(fmaf(o.x, f, w[k]), fmaf(o.y, f, w[k + 1]), fmaf(o.z, f, w[k + 2]), fmaf(o.w, f, w[k + 3]));
    }
  }
}

// PARTS: CTAs may walk more than kPartSlots slots of an item
template <int D, bool PARTS>
__global__ void __launch_bounds__(kTcThreads, 1) kv8_attend_tc_kernel(AttnArgs a) {
  using C = Tc<D>;
  constexpr int kPart = kPartSlots / kTcTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = sm + C::q;
  uint8_t* ring = sm + C::ring;
  float* mem_ref = reinterpret_cast<float*>(sm + C::mem_ref);
  int* before = reinterpret_cast<int*>(sm + C::plan);
  int* nmax = before + kMaxPlan + 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::bars);
  uint64_t *kv_full = bars, *kv_empty = bars + C::NS, *q_full = bars + 2 * C::NS, *s_full = q_full + 2,
           *p_full = q_full + 4, *o_full = q_full + 6;
  volatile int* abort_sm = reinterpret_cast<volatile int*>(q_full + 8);
  uint32_t* tmem_sm = reinterpret_cast<uint32_t*>(q_full + 8) + 1;
  __shared__ unsigned scan_sh[33];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    *abort_sm = 0;
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&kv_full[i], 4);
      mbar_init(&kv_empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 4);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&o_full[s], 1);
    }
    fence_mbar_init();
  }
  pdl_wait();
  long long u0, u1;
  int e_base;
  Cursor cur;
  if (!begin_line<kTcThreads>(a, kTcRows, kTcTile, before, nmax, scan_sh, cur, u0, u1, e_base)) return;
  if (warp == 12) {
    tmem_alloc(tmem_sm, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // (not before: a dependent that takes tensor memory first would wait for this CTA, and it for that)
  // all 512 columns are this CTA's, so they start at 0: S0, S1 at 0, 128; O0, O1
  // at 256, 256 + D
  if (*tmem_sm != 0) *abort_sm = 1;

  // every role walks the same segments: the units of the range that belong to
  // one item
  auto segment_units = [&](long long u) { return (int)min((long long)(cur.units - cur.local), u1 - u); };
  auto next_segment = [&](long long& u, int count) {
    u += max(count, 1);
    cur.local += count - 1;
    if (u < u1) cur.next(before, nmax, a.H, a.E);
  };

  if (warp < 8) {
    // -------------------------------------------------- softmax and output --
    const int st = warp >> 2, row = tid & 127;         // stream, row in it
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = lanes + st * 128, tO = lanes + 256 + st * D;
    float4* table = reinterpret_cast<float4*>(sm + C::table) + warp * 64;
    // the scale's sign goes into the queries, its size into the keys' factors: there
    // 2^-16 to 2^8 are in range whatever the exponent byte, beyond that powers of two go
    // into the queries' exponents
    const float qsign = a.scale2 < 0.f ? -1.f : 1.f;
    const int scale_e = fabsf(a.scale2) < 0x1p-126f ? 0 : (int)(__float_as_uint(fabsf(a.scale2)) >> 23) - 127;
    const int scale_q = scale_e - min(max(scale_e, -16), 8);
    const float scale_k = fabsf(a.scale2) * pow2i(-scale_q);
    int tiles = 0, segment = 0, parity_o = 0;
    bool ok = true;
    for (long long u = u0; u < u1; ++segment) {
      const int count = segment_units(u);
      const int rho = (cur.e + e_base) % a.RT * kTcRows + st * 128 + row;  // (Q G < 2^31)
      const int head = (cur.e + e_base) / a.RT * a.H + cur.h;             // (B H < 2^31)
      const int local0 = cur.local;
      const bool live = rho < a.Q * a.G;
      // rows beyond the last see everything: no tile needs a mask for them
      const int vis = live ? min(a.n_vis[(int64_t)(head / a.H) * a.Q + rho / a.G], a.N) : 0x7fffffff;
      // element of q and out that the row begins with
      auto row_at = [&]() {
        return (((int64_t)(head / a.H) * a.Q + rho / a.G) * a.H * a.G + head % a.H * a.G + rho % a.G) * D;
      };
      float qscale = 1.f;
      // of a logit; never 0, which a masked slot's -inf would turn into NaN (a scale of
      // 0, powers of two that underflow)
      auto factor = [&](float key) { return fmaf(key, qscale, 0x1p-126f); };
      if (count > 0) {
        // ---- Q: fp16 times a power of two per row, largest magnitude in [2^14, 2^15)
        const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) + (live ? row_at() : 0));
        // (read twice: held in registers it would have the loop's values spilled)
        uint32_t top = 0;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = live ? q[c] : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t m0 = (w[i] << 16) & 0x7fff0000u, m1 = w[i] & 0x7fff0000u;
            if (m0 < 0x7f800000u) top = max(top, m0);  // (infinities and NaN do not count)
            if (m1 < 0x7f800000u) top = max(top, m1);
          }
        }
        const int qe = top ? max((int)(top >> 23) - 127 - 14, -126) : 0;
        qscale = pow2i(clamp_exp(qe + scale_q));
        const float f = pow2i(-qe) * qsign;
#pragma unroll 2
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = live ? q[c] : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = pack_h2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
          *reinterpret_cast<uint4*>(sQ + st * C::row_tile + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[st]);
      }
      // the row's sum in memory, dims c to c + 3 (a warp's rows side by side)
      auto sum_at = [&](int c) { return a.sum_o + ((int64_t)blockIdx.x * (D / 4) + c / 4) * kTcRows + st * 128 + row; };
      float m = -INFINITY, mx = -INFINITY, l = 0.f;
      bool wild = false;
      // exponents of the 16-slot groups of four tiles, a lane one of each; their
      // factors go to a table four tiles at a time
      int ke = 127, ve = 127;
      auto fetch = [&](int i) {
        const int s = (local0 + i) * kTcTile + lane * 16;
        ke = ve = 127;
        if (s < cur.n) {
          const int64_t at = (int64_t)head * a.NB + (s >> a.shift);
          ke = a.k_exp[at];
          ve = a.v_exp[at];
        }
      };
      if (count > 0) fetch(0);
#pragma unroll 1
      for (int i = 0; i < count; ++i, ++tiles) {
        const int s0 = (local0 + i) * kTcTile;
        bool turn = false;
        if ((i & 3) == 0) {
          const int vl = ve - 127;
          table[(i & 4) * 8 + lane] =
              make_float4(scale_k * pow2i(clamp_exp(ke - 127)), (float)vl, pow2i(clamp_exp(-vl - (int)kTcShift)), 0.f);
          turn = !wild && __any_sync(0xffffffffu, vl < -kTame || vl > kTame);
          __syncwarp();
          if (i + 4 < count) fetch(i + 4);
        }
        const float4* tab = table + (i & 7) * 8;
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[st], tiles & 1, abort_sm))) { ok = false; break; }
        tc_fence_after();
        if (__any_sync(0xffffffffu, vis < s0 + kTcTile)) {  // masked slots: -inf, back into S
#pragma unroll 1
          for (int c = 0; c < kTcTile; c += 16) {
            float v[16];
            tmem_ld16(tS + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (s0 + c + k >= vis) v[k] = -INFINITY;
            tmem_st16(tS + c, v);
          }
          tmem_wait_st();
        }
        // ---- the largest y = x + ve (S is read here and again below: it does not
        // stay in registers)
        float tm = -INFINITY;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float v[64];
          tmem_ld32(tS + hh * 64, v);
          tmem_ld32(tS + hh * 64 + 32, v + 32);
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float4 t = tab[hh * 4 + g];
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = fmaxf(fmaxf(v[16 * g + k], v[16 * g + k + 4]), fmaxf(v[16 * g + k + 8], v[16 * g + k + 12]));
            tm = fmaxf(tm, fmaf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), factor(t.x), t.y));
          }
        }
        if (turn) {  // from here on the sum has a reference of its own
          wild = true;
          mx = m;
        }
        if (__any_sync(0xffffffffu, tm > m + kTcLazy)) {
          const float m1 = fmaxf(m, tm);
          const float f = m1 > m ? fast_exp2(m - m1) : 1.f;
          if (!wild) l *= f;
          if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {  // (S is there: the P V before it is done)
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float w[16];
              tmem_ld16(tO + c, w);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] *= f;
              tmem_st16(tO + c, w);
            }
          }
          m = m1;
        }
        if constexpr (PARTS) {
          if (i > 0 && i % kPart == 0) {  // (S is there: the P V before it is done)
            const bool begin = i == kPart;
            const float m0 = begin ? -INFINITY : mem_ref[st * 128 + row];
            const float f = m0 == -INFINITY ? 0.f : fast_exp2(m0 - m);
            mem_ref[st * 128 + row] = m;
            put_part<D>(tO, sum_at(0), f, begin);
          }
        }
        // the row's block weights from slot s0 on
        auto logs = [&]() { return a.blk_log + ((int64_t)head * a.Q * a.G + rho) * a.NSB + (s0 >> a.sub_shift); };
        if (wild) {
          // value exponents far apart: p may vanish where the sum does not
          float xm = mx;
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            const float c = tab[g].x * qscale;
            float v[16];
            tmem_ld16(tS + g * 16, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (s0 + 16 * g + k < vis) xm = fmaxf(xm, v[k] * c);
            __syncwarp();
          }
          l *= xm > mx ? fast_exp2(mx - xm) : 1.f;
          mx = xm;
          float held = 0.f;
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            const float c = tab[g].x * qscale;
            float v[16], sum = 0.f;
            tmem_ld16(tS + g * 16, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (s0 + 16 * g + k < vis) sum += fast_exp2(fmaf(v[k], c, -mx));
            l += sum;
            if (a.blk_log && live && s0 + 16 * g < vis) {
              float* blk = logs();
              if (a.sub == 16) blk[g] = log2f(sum) + mx;
              else blk[g >> 1] = log2f(held = (g & 1 ? held : 0.f) + sum) + mx;
            }
            __syncwarp();
          }
        }
        // ---- p = 2^(y - m + 7), sums by 16 slots
        const float off = m == -INFINITY ? 0.f : kTcShift - m;
        float ladd = 0.f;
#pragma unroll 1
        for (int hh = 0; hh < 4; ++hh) {
          float v[32];
          tmem_ld32(tS + hh * 32, v);
          tmem_wait_ld();
          float pk[16], sums[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float4 t = tab[2 * hh + g];
            const float tc = factor(t.x);
            const float2 c = make_float2(tc, tc), o = make_float2(t.y + off, t.y + off);
            float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float2 z = fma2(make_float2(v[16 * g + k], v[16 * g + k + 1]), c, o);
              const float2 p = ((k >> 1) % 4 == 3) ? exp2_poly(z) : make_float2(fast_exp2(z.x), fast_exp2(z.y));
              s2[(k >> 1) & 1] = add2(s2[(k >> 1) & 1], p);
              pk[g * 8 + k / 2] = __uint_as_float(pack_h2(p.x, p.y));
            }
            s2[0] = add2(s2[0], s2[1]);
            sums[g] = s2[0].x + s2[0].y;
            ladd = fmaf(sums[g], t.z, ladd);
          }
          tmem_st16(tS + hh * 16, pk);
          if (a.blk_log) {
            if (live && !wild && s0 + 32 * hh < vis) {
              float* blk = logs();
              const float b0 = off + tab[2 * hh].y, b1 = off + tab[2 * hh + 1].y;
              const bool both = s0 + 32 * hh + 16 < vis;
              if (a.sub == 32) {
                blk[hh] = log2f(sums[0] + (both ? sums[1] : 0.f)) - b0;
              } else {
                blk[2 * hh] = log2f(sums[0]) - b0;
                if (both) blk[2 * hh + 1] = log2f(sums[1]) - b1;
              }
            }
            __syncwarp();
          }
        }
        if (!wild) l += ladd;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[st]);
      }
      if (!ok) break;
      // ---- the item's rows, or this CTA's piece of them
      const bool complete = count == cur.units;
      if (!wild) mx = m;
      float inv = 0.f, gap = 0.f;  // (their product may be below fp32's range where the output is not)
      if (complete && live) {
        if (a.sink) l += fast_exp2(a.sink[head % a.H * a.G + rho % a.G] * kLog2e - mx);
        inv = 0x1p-7f / l;
        gap = fast_exp2(m - mx);
        if (a.row_log) a.row_log[(int64_t)head * a.Q * a.G + rho] = log2f(l) + mx;
      }
      if (count > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(&o_full[st], parity_o & 1, abort_sm))) break;
        ++parity_o;
        tc_fence_after();
      }
      const bool in_memory = PARTS && count > kPart;
      const float back = in_memory && mem_ref[st * 128 + row] != -INFINITY ? fast_exp2(mem_ref[st * 128 + row] - m) : 0.f;
      auto take_up = [&](int c, float (&w)[16]) {
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 o = __ldcg(sum_at(c + k));
          w[k] = fmaf(o.x, back, w[k]);
          w[k + 1] = fmaf(o.y, back, w[k + 1]);
          w[k + 2] = fmaf(o.z, back, w[k + 2]);
          w[k + 3] = fmaf(o.w, back, w[k + 3]);
        }
      };
      __syncwarp();
      if (!complete) {
        const int64_t slot = ((int64_t)blockIdx.x * 2 + (segment == 0 ? 0 : 1)) * kTcRows + st * 128 + row;
        a.part_ml[slot] = make_float4(m, mx, l, 0.f);
        float* part = a.part_o + slot * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float w[16];
          tmem_ld16(tO + c, w);
          tmem_wait_ld();
          if (PARTS && in_memory) take_up(c, w);
#pragma unroll
          for (int k = 0; k < 16; k += 4) *reinterpret_cast<float4*>(part + c + k) = make_float4(w[k], w[k + 1], w[k + 2], w[k + 3]);
        }
      } else {
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + (live ? row_at() : 0);
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float w[16];
          if (count > 0) {
            tmem_ld16(tO + c, w);
            tmem_wait_ld();
          }
          if (PARTS && in_memory) take_up(c, w);
          uint32_t o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {  // (a row that sees nothing: zeros, whatever O holds)
            const __nv_bfloat162 h2 = vis > 0 ? __floats2bfloat162_rn(w[2 * k] * inv * gap, w[2 * k + 1] * inv * gap) : __floats2bfloat162_rn(0.f, 0.f);
            o[k] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          if (live) {
            *reinterpret_cast<uint4*>(out + c) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      next_segment(u, count);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------- widen the codes --
    widen_role<D, kTcTile, C::NS>(a, cur, u0, u1, e_base, before, nmax, ring, kv_full, kv_empty, abort_sm);
  } else {
    // --------------------------------------------------------------- MMA --
    // The whole warp walks the loop on warp-uniform values and one elected lane
    // issues: descriptors stay in uniform registers (a branch on the lane costs
    // 75 cycles a product to issue, which the tensor cores do in 64).
    constexpr uint32_t idesc_qk = idesc_f16(128, kTcTile), idesc_pv = idesc_f16(128, D, true);
    const uint32_t qb = smem_u32(sQ), rb = smem_u32(ring);
    int kv = 0, tiles = 0, segs = 0;  // ring tiles and tiles of each stream so far; segments with tiles
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_sm));
      return ok;
    };
    auto wait_kv = [&](int i) { return wait(&kv_full[i % C::NS], (i / C::NS) & 1); };
    auto issue_qk = [&](int s, int i) {  // S_s = Q_s K^T, K in ring tile i
      const uint64_t qd = sdesc_k_sw128(qb + s * C::row_tile), kd = sdesc_k_sw128(rb + (i % C::NS) * C::row_tile);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t step = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;  // (the address field does not overflow)
          mma_bf16(s * 128, qd + step, kd + step, idesc_qk, k > 0);
        }
        mma_commit(&s_full[s]);
        if (s == 1) mma_commit(&kv_empty[i % C::NS]);
      }
      __syncwarp();
    };
    for (long long u = u0; ok && u < u1;) {
      const int count = __shfl_sync(0xffffffffu, segment_units(u), 0);
      if (count > 0) {
        wait_kv(kv);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!wait(&q_full[s], segs & 1)) break;
          tc_fence_after();
          issue_qk(s, kv);
        }
        ++segs;
      }
#pragma unroll 1
      for (int i = 0; ok && i < count; ++i, ++tiles, kv += 2) {
        const uint64_t vd = sdesc_mn_sw128(rb + ((kv + 1) % C::NS) * C::row_tile, 16384, 1024);
        const bool fresh = PARTS ? i % kPart == 0 : i == 0;  // O starts here
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (s == 0) wait_kv(kv + 1);
          if (!wait(&p_full[s], tiles & 1)) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kTcTile / 16; ++k)
              mma_f16_ts(256 + s * D, s * 128 + k * 8, vd + k * (2048 >> 4), idesc_pv, !fresh || k > 0);
            if (s == 1) mma_commit(&kv_empty[(kv + 1) % C::NS]);
            if (i + 1 == count) mma_commit(&o_full[s]);
          }
          __syncwarp();
          if (i + 1 < count) {
            if (s == 0 && !wait_kv(kv + 2)) break;
            tc_fence_after();
            issue_qk(s, kv + 2);
          }
        }
      }
      next_segment(u, count);
    }
  }
  if (*abort_sm && lane == 0) {
    atomicOr(a.err, CSA_DEV_TIMEOUT);
    const uint64_t t0 = globaltimer();  // products already issued end before TMEM is given back
    while (globaltimer() - t0 < 200000ull) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(*tmem_sm, 512);
}

template <int D>
csa_status launch_tc(AttnArgs& a, cudaStream_t st) {
  auto kern = a.parts ? kv8_attend_tc_kernel<D, true> : kv8_attend_tc_kernel<D, false>;
  const int smem = Tc<D>::total + 1024;
  if (!set_kernel_smem((const void*)kern, smem)) return CSA_ERR_CUDA;
  const long long items = (long long)a.E * a.H;
  long long grid = items;
  if (a.planned) {
    const long long units = items * ((a.N + kTcTile - 1) / kTcTile);
    grid = sm_count() < kMaxGrid ? sm_count() : kMaxGrid;
    if (units < grid) grid = units;
  }
  if (items * (kTcRows / kTcJoinRows) > 0x7fffffffll || (long long)a.Q * a.G + kTcRows > 0x7fffffffll ||
      (long long)a.B * a.H > 0x7fffffffll)
    return CSA_ERR_SHAPE;
  csa_status ok = CSA_OK;
  CSA_LAUNCH(KK_KV8_ATTEND_TC, st,
             if (launch_maybe_pdl(true, kern, dim3((unsigned)grid), dim3(kTcThreads), smem, st, a) !=
                 cudaSuccess) ok = CSA_ERR_CUDA);
  if (a.planned)
    CSA_LAUNCH(KK_KV8_COMBINE, st,
               if (launch_maybe_pdl(true, (kv8_join<__nv_bfloat16, D, kTcRows>), dim3((unsigned)(items * (kTcRows / kTcJoinRows))),
                                    dim3(256), 0, st, a, (int)grid) != cudaSuccess) ok = CSA_ERR_CUDA);
  return ok != CSA_OK ? ok : last_launch_status();
}

}  // namespace

int kv8_attend_tc_rows() { return kTcRows; }

csa_status launch_kv8_attend_tc(const csa_kv8_params& p, AttnArgs& a, cudaStream_t st) {
  return p.d == 64 ? launch_tc<64>(a, st) : launch_tc<128>(a, st);
}

}  // namespace csa
