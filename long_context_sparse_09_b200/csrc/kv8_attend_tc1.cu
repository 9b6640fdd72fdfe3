// kv8_attend_tc1.cu -- attention over the 8-bit KV cache for many query rows a
// KV head, fp32 activations or d = 256 or calls too small for CTAs of 256 rows,
// on the 5th-generation tensor cores.
//
// The mathematics is that of kv8_attend_tc.cu.  fp32 queries and probabilities
// are two fp16 terms each, so both products run twice; two streams of 128 rows
// then fit neither shared nor tensor memory, and O of 256 dims does not either.
// A CTA owns 128 query rows: its two softmax warpgroups take the tiles of slots
// in turn (S in two buffers), so that Q K^T of the next tile and the softmax of
// two tiles overlap.  Both add to one O, so they share its reference M (row by
// row in shared memory): a warpgroup reads what the other one left, raises it
// where its tile needs that (and rescales O, after the last P V), and passes it
// on before it forms P.  Sums stay with their warpgroup until the end.
//
// What bounds it: the softmax of a tile (about 3,000 cycles of one warpgroup, two
// of them running) against its products.  The last 2048 queries over 8K slots, 64
// heads, 8 KV heads (cache not in L2): bf16, d = 256 1.18 ms (810 TFLOP/s); fp32, d = 128
// 1.08 ms (450 TFLOP/s of fp32 attention, twice that in fp16 products; 14% of it the
// sums in parts), d = 64 0.82 ms, d = 256, with room for one K and one V tile only,
// 2.84 ms; on mma.sync (kv8_attend.cu; cache in L2) 5.2, 3.25, 2.25 and 6.7 ms.
#include "kv8_attend_tc.cuh"

namespace csa {

using namespace kv8;

namespace {

constexpr int kTc1Rows = 128;  // query rows of a CTA

template <typename T, int D, bool PARTS>
struct Tc1 {
  static constexpr int SPLIT = sizeof(T) == 4 ? 2 : 1;  // fp16 terms of q and p
  static constexpr int KT = D == 256 ? 64 : 128;        // slots of a tile
  static constexpr int NG = KT / 16;
  // fp32: after so many tiles (2048 slots; even) O is added to the row's sum in
  // memory and starts anew.  The tensor cores cut off what they add to an
  // accumulator, always towards zero: over 16K slots O shrank by 1.4e-5 (relative
  // error 1.7e-5; with the parts 4.4e-6, with parts of 1024 slots 3.1e-6, plain fp32
  // torch 2.6e-6).  It costs 14% (d = 128; parts of 1024: 24%).
  // bf16: where CTAs may walk more than kPartSlots slots of an item, after those.
  static constexpr int flush = SPLIT == 2 ? 2048 / KT : PARTS ? kPartSlots / KT : 0;
  static constexpr int q_term = kTc1Rows * D * 2;       // a term of the queries
  static constexpr int kv_tile = KT * D * 2;            // a K or V tile in fp16
  static constexpr int NS = D == 64 ? 8 : D == 256 && SPLIT == 2 ? 2 : 4;  // of them in the ring
  static constexpr int q = 0;
  static constexpr int ring = SPLIT * q_term;
  static constexpr int table = ring + NS * kv_tile;     // [8 warps][2][NG] float4
  static constexpr int ref = table + 8 * 2 * NG * 16;   // [128] M of O
  static constexpr int mem_ref = ref + kTc1Rows * 4;    // [128] M of the rows' sums in memory
  static constexpr int pair = mem_ref + kTc1Rows * 4;       // [2][128] a warpgroup's reference of its sum, sum
  static constexpr int plan = pair + 2 * kTc1Rows * 8;  // units before, n_max: [E + 1], [E]
  static constexpr int bars = plan + (2 * kMaxPlan + 2) * 4;
  static constexpr int total = bars + (2 * NS + 10) * 8 + 16;
  static_assert(total + 1024 <= 232448, "shared memory");
  // tensor memory: S of the two buffers (P's first term over their front), O, P's
  // second term
  static constexpr int colO = 2 * KT, colP2 = colO + D;
  static_assert(colP2 + (SPLIT - 1) * KT <= 512, "tensor memory");
};

template <typename T, int D, bool PARTS>
__global__ void __launch_bounds__(kTcThreads, 1) kv8_attend_tc1_kernel(AttnArgs a) {
  using C = Tc1<T, D, PARTS>;
  constexpr int KT = C::KT, SPLIT = C::SPLIT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = sm + C::q;
  uint8_t* ring = sm + C::ring;
  float* ref = reinterpret_cast<float*>(sm + C::ref);
  float* mem_ref = reinterpret_cast<float*>(sm + C::mem_ref);
  float2* pair = reinterpret_cast<float2*>(sm + C::pair);
  int* before = reinterpret_cast<int*>(sm + C::plan);
  int* nmax = before + kMaxPlan + 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::bars);
  uint64_t *kv_full = bars, *kv_empty = bars + C::NS, *s_full = bars + 2 * C::NS, *p_full = s_full + 2,
           *pv_done = s_full + 4, *turn = s_full + 6, *q_full = s_full + 8, *fin = s_full + 9;
  volatile int* abort_sm = reinterpret_cast<volatile int*>(s_full + 10);
  uint32_t* tmem_sm = reinterpret_cast<uint32_t*>(s_full + 10) + 1;
  __shared__ unsigned scan_sh[33];
  __shared__ int wild_sm[4];  // by 32 rows: the last segment (from 1) with value exponents far apart
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid < 4) wild_sm[tid] = 0;
  if (tid == 0) {
    *abort_sm = 0;
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&kv_full[i], 4);
      mbar_init(&kv_empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&pv_done[s], 1);
      mbar_init(&turn[s], 4);
    }
    mbar_init(q_full, 8);
    mbar_init(fin, 8);
    fence_mbar_init();
  }
  pdl_wait();
  long long u0, u1;
  int e_base;
  Cursor cur;
  if (!begin_line<kTcThreads>(a, kTc1Rows, KT, before, nmax, scan_sh, cur, u0, u1, e_base)) return;
  if (warp == 12) {
    tmem_alloc(tmem_sm, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // (not before: a dependent that takes tensor memory first would wait for this CTA, and it for that)
  // all 512 columns are this CTA's, so they start at 0
  if (*tmem_sm != 0) *abort_sm = 1;

  auto segment_units = [&](long long u) { return (int)min((long long)(cur.units - cur.local), u1 - u); };
  auto next_segment = [&](long long& u, int count) {
    u += max(count, 1);
    cur.local += count - 1;
    if (u < u1) cur.next(before, nmax, a.H, a.E);
  };

  if (warp < 8) {
    // -------------------------------------------------- softmax and output --
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = lanes + wg * KT, tP2 = lanes + C::colP2 + wg * (KT / 2), tO = lanes + C::colO;
    float4* table = reinterpret_cast<float4*>(sm + C::table) + warp * 2 * C::NG;
    // the scale's sign goes into the queries, its size into the keys' factors: there
    // 2^-16 to 2^8 are in range whatever the exponent byte, beyond that powers of two go
    // into the queries' exponents
    const float qsign = a.scale2 < 0.f ? -1.f : 1.f;
    const int scale_e = fabsf(a.scale2) < 0x1p-126f ? 0 : (int)(__float_as_uint(fabsf(a.scale2)) >> 23) - 127;
    const int scale_q = scale_e - min(max(scale_e, -16), 8);
    const float scale_k = fabsf(a.scale2) * pow2i(-scale_q);
    int tile0 = 0, turns = 0, segs = 0, segment = 0;  // tiles before the segment, of both warpgroups
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity & 1, abort_sm)) != 0;
    };
    for (long long u = u0; u < u1; ++segment) {
      const int count = segment_units(u);
      const int rho = (cur.e + e_base) % a.RT * kTc1Rows + row;  // (Q G < 2^31)
      const int head = (cur.e + e_base) / a.RT * a.H + cur.h;   // (B H < 2^31)
      const int local0 = cur.local;
      const bool live = rho < a.Q * a.G;
      // rows beyond the last see everything: no tile needs a mask for them
      const int vis = live ? min(a.n_vis[(int64_t)(head / a.H) * a.Q + rho / a.G], a.N) : 0x7fffffff;
      auto row_at = [&]() {
        return (((int64_t)(head / a.H) * a.Q + rho / a.G) * a.H * a.G + head % a.H * a.G + rho % a.G) * D;
      };
      float qscale = 1.f;
      // of a logit; never 0, which a masked slot's -inf would turn into NaN (a scale of
      // 0, powers of two that underflow)
      auto factor = [&](float key) { return fmaf(key, qscale, 0x1p-126f); };
      if (count > 0) {
        // ---- Q: fp16 terms times a power of two per row, largest magnitude in
        // [2^14, 2^15); a warpgroup writes half of the dims
        const T* q = reinterpret_cast<const T*>(a.q) + (live ? row_at() : 0);
        uint32_t top = 0;
#pragma unroll 4
        for (int c = 0; c < D; c += 16 / (int)sizeof(T)) {
          const uint4 v = live ? *reinterpret_cast<const uint4*>(q + c) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (SPLIT == 2) {
              const uint32_t m0 = w[i] & 0x7fffffffu;
              if (m0 < 0x7f800000u) top = max(top, m0);  // (infinities and NaN do not count)
            } else {
              const uint32_t m0 = (w[i] << 16) & 0x7fff0000u, m1 = w[i] & 0x7fff0000u;
              if (m0 < 0x7f800000u) top = max(top, m0);
              if (m1 < 0x7f800000u) top = max(top, m1);
            }
          }
        }
        const int qe = top ? max((int)(top >> 23) - 127 - 14, -126) : 0;
        qscale = pow2i(clamp_exp(qe + scale_q));
        const float f = pow2i(-qe) * qsign;
#pragma unroll 2
        for (int c8 = wg * (D / 16); c8 < (wg + 1) * (D / 16); ++c8) {  // 8 dims
          float x[8];
          if constexpr (SPLIT == 2) {
            const float4 v0 = live ? *reinterpret_cast<const float4*>(q + c8 * 8) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 v1 = live ? *reinterpret_cast<const float4*>(q + c8 * 8 + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
            x[0] = v0.x; x[1] = v0.y; x[2] = v0.z; x[3] = v0.w;
            x[4] = v1.x; x[5] = v1.y; x[6] = v1.z; x[7] = v1.w;
          } else {
            const uint4 v = live ? *reinterpret_cast<const uint4*>(q + c8 * 8) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[2 * i] = __uint_as_float(w[i] << 16);
              x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
          }
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float y0 = x[2 * i] * f, y1 = x[2 * i + 1] * f;
            hi[i] = pack_h2(y0, y1);
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi[i]));
            lo[i] = pack_h2(y0 - h.x, y1 - h.y);
          }
          uint8_t* dst = sQ + (c8 >> 3) * (kTc1Rows * 128) + row * 128 + (((c8 & 7) ^ (row & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          if constexpr (SPLIT == 2) *reinterpret_cast<uint4*>(dst + C::q_term) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      const bool complete = count == cur.units;
      const int64_t slot = ((int64_t)blockIdx.x * 2 + (segment == 0 ? 0 : 1)) * kTc1Rows + row;
      // where the row's sum goes: the output, or this CTA's piece of it
      T* out = reinterpret_cast<T*>(a.out) + (live ? row_at() : 0);
      float* part = a.part_o + slot * D;
      // fp32: the sum of the row's parts lies there as well; bf16: in memory of its own
      auto sum_of_parts = [&]() {
        if constexpr (SPLIT == 2)
          return complete ? reinterpret_cast<float*>(out) : part;
        else
          return reinterpret_cast<float*>(a.sum_o) + ((int64_t)blockIdx.x * kTc1Rows + row) * D;
      };
      float m = -INFINITY, mx = -INFINITY, l = 0.f;
      bool wild = false;
      // The reference that the other warpgroup left, m0 >= m.  Value exponents far apart
      // that only its tiles hold may have lifted it: this one's sum, which is of x, then
      // keeps a reference of its own as well (under m0 it could vanish, next to the
      // least of exp2_poly).
      auto follow = [&]() {
        const float m0 = ref[row];
        if (!wild && wild_sm[warp & 3] == segment + 1) {
          wild = true;
          mx = m;
        }
        if (m0 != m) {  // (m0 > m; m = -inf: l is 0)
          if (!wild) l *= fast_exp2(m - m0);
          m = m0;
        }
      };
      // exponents of a tile's 16-slot groups: lanes 0 .. NG - 1 hold one of each
      int ke = 127, ve = 127;
      auto fetch = [&](int i) {
        const int s = (local0 + i) * KT + (lane & (C::NG - 1)) * 16;
        ke = ve = 127;
        if (s < cur.n) {
          const int64_t at = (int64_t)head * a.NB + (s >> a.shift);
          ke = a.k_exp[at];
          ve = a.v_exp[at];
        }
      };
      const int mine = (tile0 ^ wg) & 1;  // this warpgroup's first tile of the segment
      if (mine < count) fetch(mine);
#pragma unroll 1
      for (int i = mine; i < count; i += 2) {
        const int s0 = (local0 + i) * KT, tile = tile0 + i;  // (tile & 1 == wg)
        float4* tab = table + (tile >> 1 & 1) * C::NG;
        const int vl = ve - 127;
        if (lane < C::NG)
          tab[lane] = make_float4(scale_k * pow2i(clamp_exp(ke - 127)), (float)vl, pow2i(clamp_exp(-vl - (int)kTcShift)), 0.f);
        const bool far = !wild && __any_sync(0xffffffffu, vl < -kTame || vl > kTame);
        __syncwarp();
        if (i + 2 < count) fetch(i + 2);
        if (!wait(&s_full[wg], tile >> 1)) { ok = false; break; }
        tc_fence_after();
        if (__any_sync(0xffffffffu, vis < s0 + KT)) {  // masked slots: -inf, back into S
#pragma unroll 1
          for (int c = 0; c < KT; c += 16) {
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
        // ---- the largest y = x + ve
        float tm = -INFINITY;
#pragma unroll
        for (int hh = 0; hh < KT / 64; ++hh) {
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
        if (far) {  // from here on the sum has a reference of its own
          wild = true;
          mx = m;
          if (lane == 0) wild_sm[warp & 3] = segment + 1;
        }
        // ---- the reference that the other warpgroup left with the tile before
        if (i > 0) {
          if (!wait(&turn[wg], turns++)) { ok = false; break; }
          follow();
        }
        if (__any_sync(0xffffffffu, tm > m + kTcLazy)) {
          const float m1 = fmaxf(m, tm);
          const float f = m1 > m ? fast_exp2(m - m1) : 1.f;
          if (!wild) l *= f;
          if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
            // (S of this tile was there, so the P V two before it is done)
            if (!wait(&pv_done[wg ^ 1], (tile - 1) >> 1)) { ok = false; break; }
            tc_fence_after();
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
        if constexpr (C::flush > 0) {
          if (i > 0 && i % C::flush == 0) {  // (the same warpgroup every time)
            if (!wait(&pv_done[wg ^ 1], (tile - 1) >> 1)) { ok = false; break; }
            tc_fence_after();
            tmem_wait_st();  // O may just have been rescaled
            // The sum keeps the reference it began with, so that adding needs no
            // answer from memory: one thread adds to an address, in its order.  Only
            // where that reference is not in reach the sum is read and scaled.
            const bool begin = i == C::flush;
            float m0 = begin ? m : mem_ref[row];
            const bool scaled = m - m0 > 60.f || m0 == -INFINITY;
            const float f = m0 == -INFINITY ? 0.f : fast_exp2(scaled ? m0 - m : m - m0);
            if (begin || scaled) mem_ref[row] = m;
            float* sum = sum_of_parts();
            __syncwarp();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float w[16];
              tmem_ld16(tO + c, w);
              tmem_wait_ld();
              if (live || !complete) {
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                  float4* at = reinterpret_cast<float4*>(sum + c + k);
                  if (begin) {
                    *at = make_float4(w[k], w[k + 1], w[k + 2], w[k + 3]);
                  } else if (scaled) {
                    const float4 o = __ldcg(at);
                    *at = make_float4(fmaf(o.x, f, w[k]), fmaf(o.y, f, w[k + 1]), fmaf(o.z, f, w[k + 2]), fmaf(o.w, f, w[k + 3]));
                  } else {
                    atomicAdd(at, make_float4(w[k] * f, w[k + 1] * f, w[k + 2] * f, w[k + 3] * f));
                  }
                }
              }
              __syncwarp();  // (rows differ above; the whole warp reads tensor memory)
            }
            tc_fence_before();
          }
        }
        ref[row] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(&turn[wg ^ 1]);
        // the row's block weights from slot s0 on
        auto logs = [&]() { return a.blk_log + ((int64_t)head * a.Q * a.G + rho) * a.NSB + (s0 >> a.sub_shift); };
        if (wild) {
          // value exponents far apart: p may vanish where the sum does not
          float xm = mx;
#pragma unroll 1
          for (int g = 0; g < C::NG; ++g) {
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
          for (int g = 0; g < C::NG; ++g) {
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
        for (int hh = 0; hh < KT / 32; ++hh) {
          float v[32];
          tmem_ld32(tS + hh * 32, v);
          tmem_wait_ld();
          float pk[16], pl[16], sums[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float4 t = tab[2 * hh + g];
            const float tc = factor(t.x);
            const float2 c = make_float2(tc, tc), o = make_float2(t.y + off, t.y + off);
            float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float2 z = fma2(make_float2(v[16 * g + k], v[16 * g + k + 1]), c, o);
              // (the polynomial's 2.9e-6 is too much for two terms of fp16)
              const float2 p = SPLIT == 1 && (k >> 1) % 4 == 3 ? exp2_poly(z) : make_float2(fast_exp2(z.x), fast_exp2(z.y));
              s2[(k >> 1) & 1] = add2(s2[(k >> 1) & 1], p);
              const uint32_t hi = pack_h2(p.x, p.y);
              pk[g * 8 + k / 2] = __uint_as_float(hi);
              if constexpr (SPLIT == 2) {
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                pl[g * 8 + k / 2] = __uint_as_float(pack_h2(p.x - h.x, p.y - h.y));
              }
            }
            s2[0] = add2(s2[0], s2[1]);
            sums[g] = s2[0].x + s2[0].y;
            ladd = fmaf(sums[g], t.z, ladd);
          }
          tmem_st16(tS + hh * 16, pk);
          if constexpr (SPLIT == 2) tmem_st16(tP2 + hh * 16, pl);
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
        if (lane == 0) mbar_arrive(&p_full[wg]);
      }
      if (!ok) break;
      // ---- the two sums become one
      if (count > 0) {
        const int last = tile0 + count - 1;
        if ((last & 1) != wg) {  // the other warpgroup had the last word on the reference
          if (!wait(&turn[wg], turns++)) break;
          follow();
        }
        if (!wild) mx = m;
        pair[wg * kTc1Rows + row] = make_float2(mx, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(fin);
        if (!wait(fin, segs++)) break;
        const float2 other = pair[(wg ^ 1) * kTc1Rows + row];
        const float top = fmaxf(mx, other.x);
        // (warpgroup 0's part first in both: the two halves of a row get the same sum)
        const float l0 = wg == 0 ? l : other.y, l1 = wg == 0 ? other.y : l;
        const float x0 = wg == 0 ? mx : other.x, x1 = wg == 0 ? other.x : mx;
        l = (x0 == -INFINITY ? 0.f : l0 * fast_exp2(x0 - top)) + (x1 == -INFINITY ? 0.f : l1 * fast_exp2(x1 - top));
        mx = top;
        if (!wait(&pv_done[last & 1], last >> 1)) break;
        tc_fence_after();
        tile0 += count;
      }
      float inv = 0.f, gap = 0.f;  // (their product may be below fp32's range where the output is not)
      if (complete && live) {
        if (a.sink) l += fast_exp2(a.sink[head % a.H * a.G + rho % a.G] * kLog2e - mx);
        inv = 0x1p-7f / l;
        gap = fast_exp2(m - mx);
        if (a.row_log && wg == 0) a.row_log[(int64_t)head * a.Q * a.G + rho] = log2f(l) + mx;
      }
      // ---- the item's rows, or this CTA's piece of them: half of the dims each
      if (!complete && wg == 0) a.part_ml[slot] = make_float4(m, mx, l, 0.f);
      const bool in_memory = C::flush > 0 && count > C::flush;
      const float m0 = in_memory ? mem_ref[row] : -INFINITY;
      const float back = m0 == -INFINITY ? 0.f : fast_exp2(m0 - m);
      __syncwarp();
#pragma unroll 1
      for (int c = wg * (D / 2); c < (wg + 1) * (D / 2); c += 16) {
        float w[16];
        if (count > 0) {
          tmem_ld16(tO + c, w);
          tmem_wait_ld();
        }
        if (in_memory && (live || !complete)) {
          const float* sum = sum_of_parts();
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            const float4 o = __ldcg(reinterpret_cast<const float4*>(sum + c + k));
            w[k] = fmaf(o.x, back, w[k]);
            w[k + 1] = fmaf(o.y, back, w[k + 1]);
            w[k + 2] = fmaf(o.z, back, w[k + 2]);
            w[k + 3] = fmaf(o.w, back, w[k + 3]);
          }
        }
        if (!complete) {
#pragma unroll
          for (int k = 0; k < 16; k += 4) *reinterpret_cast<float4*>(part + c + k) = make_float4(w[k], w[k + 1], w[k + 2], w[k + 3]);
        } else if (live) {
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = vis > 0 ? w[k] * inv * gap : 0.f;  // (a row that sees nothing: whatever O holds)
          if constexpr (SPLIT == 2) {
#pragma unroll
            for (int k = 0; k < 16; k += 4) *reinterpret_cast<float4*>(out + c + k) = make_float4(w[k], w[k + 1], w[k + 2], w[k + 3]);
          } else {
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(w[2 * k], w[2 * k + 1]);
              o[k] = *reinterpret_cast<const uint32_t*>(&h2);
            }
            *reinterpret_cast<uint4*>(out + c) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      next_segment(u, count);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------- widen the codes --
    widen_role<D, KT, C::NS>(a, cur, u0, u1, e_base, before, nmax, ring, kv_full, kv_empty, abort_sm);
  } else {
    // --------------------------------------------------------------- MMA --
    // (the whole warp on uniform values, one elected lane issues)
    constexpr uint32_t idesc_qk = idesc_f16(128, KT), idesc_pv = idesc_f16(128, D, true);
    const uint32_t qb = smem_u32(sQ), rb = smem_u32(ring);
    int kv = 0, tile = 0, segs = 0;  // ring tiles, tiles so far; segments with tiles
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity & 1, abort_sm));
      return ok;
    };
    auto issue_qk = [&](int i, int buf) {  // S = Q K^T, K in ring tile i
      if (!wait(&kv_full[i % C::NS], i / C::NS)) return;
      tc_fence_after();
      const uint64_t qd = sdesc_k_sw128(qb), kd = sdesc_k_sw128(rb + (i % C::NS) * C::kv_tile);
      if (elect_one()) {
#pragma unroll
        for (int t = 0; t < SPLIT; ++t)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)  // (the address fields do not overflow)
            mma_bf16(buf * KT, qd + ((t * C::q_term + (k >> 2) * (kTc1Rows * 128) + (k & 3) * 32) >> 4),
                     kd + (((k >> 2) * (KT * 128) + (k & 3) * 32) >> 4), idesc_qk, t > 0 || k > 0);
        mma_commit(&s_full[buf]);
        mma_commit(&kv_empty[i % C::NS]);
      }
      __syncwarp();
    };
    for (long long u = u0; ok && u < u1;) {
      const int count = __shfl_sync(0xffffffffu, segment_units(u), 0);
      if (count > 0 && wait(q_full, segs++)) issue_qk(kv, tile & 1);
#pragma unroll 1
      for (int i = 0; ok && i < count; ++i, ++tile, kv += 2) {
        const int buf = tile & 1;
        if (i + 1 < count) issue_qk(kv + 2, buf ^ 1);
        if (!wait(&kv_full[(kv + 1) % C::NS], (kv + 1) / C::NS) || !wait(&p_full[buf], tile >> 1)) break;
        tc_fence_after();
        const uint64_t vd = sdesc_mn_sw128(rb + ((kv + 1) % C::NS) * C::kv_tile, KT * 128, 1024);
        const bool fresh = C::flush > 0 ? i % (C::flush > 0 ? C::flush : 1) == 0 : i == 0;  // O starts here
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < KT / 16; ++k) {
            mma_f16_ts(C::colO, buf * KT + k * 8, vd + k * (2048 >> 4), idesc_pv, !fresh || k > 0);
            if constexpr (SPLIT == 2)
              mma_f16_ts(C::colO, C::colP2 + buf * (KT / 2) + k * 8, vd + k * (2048 >> 4), idesc_pv, 1);
          }
          mma_commit(&pv_done[buf]);
          mma_commit(&kv_empty[(kv + 1) % C::NS]);
        }
        __syncwarp();
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

template <typename T, int D, bool PARTS>
csa_status launch_tc1(AttnArgs& a, cudaStream_t st) {
  auto kern = kv8_attend_tc1_kernel<T, D, PARTS>;
  const int smem = Tc1<T, D, PARTS>::total + 1024;
  if (!set_kernel_smem((const void*)kern, smem)) return CSA_ERR_CUDA;
  const long long items = (long long)a.E * a.H;
  long long grid = items;
  if (a.planned) {
    const long long units = items * ((a.N + Tc1<T, D, PARTS>::KT - 1) / Tc1<T, D, PARTS>::KT);
    grid = sm_count() < kMaxGrid ? sm_count() : kMaxGrid;
    if (units < grid) grid = units;
  }
  if (items * (kTc1Rows / kTcJoinRows) > 0x7fffffffll || (long long)a.Q * a.G + kTc1Rows > 0x7fffffffll ||
      (long long)a.B * a.H > 0x7fffffffll)
    return CSA_ERR_SHAPE;
  csa_status ok = CSA_OK;
  CSA_LAUNCH(KK_KV8_ATTEND_TC1, st,
             if (launch_maybe_pdl(true, kern, dim3((unsigned)grid), dim3(kTcThreads), smem, st, a) !=
                 cudaSuccess) ok = CSA_ERR_CUDA);
  if (a.planned)
    CSA_LAUNCH(KK_KV8_COMBINE, st,
               if (launch_maybe_pdl(true, (kv8_join<T, D, kTc1Rows>),
                                    dim3((unsigned)(items * (kTc1Rows / kTcJoinRows))), dim3(256), 0, st, a,
                                    (int)grid) != cudaSuccess) ok = CSA_ERR_CUDA);
  return ok != CSA_OK ? ok : last_launch_status();
}

}  // namespace

int kv8_attend_tc1_rows() { return kTc1Rows; }

csa_status launch_kv8_attend_tc1(const csa_kv8_params& p, AttnArgs& a, cudaStream_t st) {
  if (p.act == CSA_F32)
    return p.d == 64    ? launch_tc1<float, 64, false>(a, st)
           : p.d == 128 ? launch_tc1<float, 128, false>(a, st)
                        : launch_tc1<float, 256, false>(a, st);
  if (a.parts)
    return p.d == 64    ? launch_tc1<__nv_bfloat16, 64, true>(a, st)
           : p.d == 128 ? launch_tc1<__nv_bfloat16, 128, true>(a, st)
                        : launch_tc1<__nv_bfloat16, 256, true>(a, st);
  return p.d == 64    ? launch_tc1<__nv_bfloat16, 64, false>(a, st)
         : p.d == 128 ? launch_tc1<__nv_bfloat16, 128, false>(a, st)
                      : launch_tc1<__nv_bfloat16, 256, false>(a, st);
}

}  // namespace csa
