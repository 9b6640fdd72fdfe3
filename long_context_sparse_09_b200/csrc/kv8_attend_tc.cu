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
//   P_s = 2^(y - M + 11) by stream s's warpgroup, a thread a row: S is read
//         from TMEM once, P (fp16) goes back over the front half of S
//   O_s += P_s V       tcgen05.mma, P from TMEM, V MN-major in shared memory
// While a stream's softmax runs, the tensor cores work for the other one.  A
// third warpgroup widens the codes: 16-byte global loads (a tile ahead, in
// registers) -> fp16 in the 128-byte swizzle layout, K and V tiles alternating
// in one ring; that costs each CTA a conversion of the tile, 1/256 of its
// products.  All tiles of the call lie on one line, cut evenly over the SMs;
// the pieces of items that several CTAs share are joined by kv8_join.
#include "kv8_attend.cuh"

namespace csa {

using namespace sm100;
using namespace kv8;

namespace {

constexpr int kTcRows = 256;     // query rows of a CTA: two streams of 128
constexpr int kTcTile = 128;     // slots of a tile
constexpr int kTcThreads = 512;  // 2 softmax warpgroups, 1 that widens, 1 for the MMA warp
constexpr int kJoinRows = 32;    // rows of a join CTA

template <int D>
struct Tc {
  static constexpr int row_tile = kTcTile * D * 2;   // 128 rows of fp16: a stream's Q, a K or V tile
  static constexpr int NS = D == 64 ? 8 : 4;         // K and V tiles in the ring
  static constexpr int q = 0;
  static constexpr int ring = 2 * row_tile;
  static constexpr int table = ring + NS * row_tile;           // [8 warps][2][8] float4
  static constexpr int plan = table + 8 * 2 * 8 * 16;          // units before, n_max: [E + 1], [E]
  static constexpr int bars = plan + (2 * kMaxPlan + 2) * 4;
  static constexpr int total = bars + (2 * NS + 8) * 8 + 16;
};

template <int kRegs> __device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs> __device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {  // codes: not kept in L1
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p));
  return v;
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) kv8_attend_tc_kernel(AttnArgs a) {
  using C = Tc<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = sm + C::q;
  uint8_t* ring = sm + C::ring;
  int* before = reinterpret_cast<int*>(sm + C::plan);
  int* nmax = before + kMaxPlan + 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::bars);
  uint64_t *kv_full = bars, *kv_empty = bars + C::NS, *q_full = bars + 2 * C::NS, *s_full = q_full + 2,
           *p_full = q_full + 4, *o_full = q_full + 6;
  volatile int* abort_sm = reinterpret_cast<volatile int*>(q_full + 8);
  uint32_t* tmem_sm = reinterpret_cast<uint32_t*>(q_full + 8) + 1;
  __shared__ unsigned scan_sh[33];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  pdl_trigger();
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
  const uint32_t tbase = *tmem_sm;  // S0, S1: columns 0, 128; O0, O1: 256, 256 + D

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
    regs_inc<192>();
    const int st = warp >> 2, row = tid & 127;         // stream, row in it
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + lanes + st * 128, tO = tbase + lanes + 256 + st * D;
    float4* table = reinterpret_cast<float4*>(sm + C::table) + warp * 16;
    const float qsign = a.scale2 < 0.f ? -1.f : 1.f, ascale = fabsf(a.scale2);
    int tiles = 0, segment = 0, parity_o = 0;
    bool ok = true;
    for (long long u = u0; u < u1; ++segment) {
      const int count = segment_units(u);
      const int h = cur.h, b = (cur.e + e_base) / a.RT, rt = (cur.e + e_base) % a.RT;
      const int local0 = cur.local, n_max = cur.n;
      const bool complete = count == cur.units;
      const int64_t head = (int64_t)b * a.H + h;
      const int64_t rho = (int64_t)rt * kTcRows + st * 128 + row;
      const bool live = rho < (int64_t)a.Q * a.G;
      const int j = live ? (int)(rho / a.G) : 0, hq = h * a.G + (int)(rho % a.G);
      const int64_t qrow = ((int64_t)b * a.Q + j) * a.H * a.G + hq;
      // rows beyond the last see everything: no tile needs a mask for them
      const int vis = live ? min(a.n_vis[(int64_t)b * a.Q + j], a.N) : 0x7fffffff;
      float qscale = 1.f;
      if (count > 0) {
        // ---- Q: fp16 times a power of two per row, largest magnitude in [2^14, 2^15)
        const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) + qrow * D);
        uint4 raw[D / 8];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          raw[c] = live ? q[c] : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t m0 = (w[i] << 16) & 0x7fff0000u, m1 = w[i] & 0x7fff0000u;
            if (m0 < 0x7f800000u) top = max(top, m0);  // (infinities and NaN do not count)
            if (m1 < 0x7f800000u) top = max(top, m1);
          }
        }
        const int qe = top ? max((int)(top >> 23) - 127 - 14, -126) : 0;
        qscale = pow2i(qe);
        const float f = pow2i(-qe) * qsign;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
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
      float m = -INFINITY, mx = -INFINITY, l = 0.f;
      bool wild = false;
      // exponents of the tile's 16-slot groups: lanes 0-7 hold one of each
      const uint8_t* ke_p = a.k_exp + head * a.NB;
      const uint8_t* ve_p = a.v_exp + head * a.NB;
      int ke = 127, ve = 127;
      auto fetch = [&](int i) {
        const int s = (local0 + i) * kTcTile + (lane & 7) * 16;
        ke = ve = 127;
        if (s < n_max) {
          ke = ke_p[s >> a.shift];
          ve = ve_p[s >> a.shift];
        }
      };
      if (count > 0) fetch(0);
#pragma unroll 1
      for (int i = 0; i < count; ++i, ++tiles) {
        const int s0 = (local0 + i) * kTcTile;
        float4* tab = table + (tiles & 1) * 8;
        const int vl = ve - 127;
        if (lane < 8) tab[lane] = make_float4(ascale * pow2i(clamp_exp(ke - 127)), (float)vl, pow2i(clamp_exp(-vl - 11)), 0.f);
        const bool turn = !wild && __any_sync(0xffffffffu, vl < -kTame || vl > kTame);
        __syncwarp();
        if (i + 1 < count) fetch(i + 1);
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[st], tiles & 1, abort_sm))) { ok = false; break; }
        tc_fence_after();
        float s[kTcTile];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s + c * 32);
        tmem_wait_ld();
        // ---- y = x + ve (kept as s, factor and offset), its maximum
        if (__any_sync(0xffffffffu, vis < s0 + kTcTile)) {
#pragma unroll
          for (int k = 0; k < kTcTile; ++k)
            if (s0 + k >= vis) s[k] = -INFINITY;
        }
        float tm = -INFINITY;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float4 t = tab[g];
          float top = s[16 * g];
#pragma unroll
          for (int k = 1; k < 16; ++k) top = fmaxf(top, s[16 * g + k]);
          tm = fmaxf(tm, fmaf(top, t.x * qscale, t.y));
        }
        if (turn) {  // from here on the sum has a reference of its own
          wild = true;
          mx = m;
        }
        if (__any_sync(0xffffffffu, tm > m + kLazy)) {
          const float m1 = fmaxf(m, tm);
          const float f = m1 > m ? fast_exp2(m - m1) : 1.f;
          if (!wild) l *= f;
          if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {  // (S is there: the P V before it is done)
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float v[16];
              tmem_ld16(tO + c, v);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] *= f;
              tmem_st16(tO + c, v);
            }
          }
          m = m1;
        }
        float* blk = nullptr;
        if (a.blk_log && live && vis > s0) blk = a.blk_log + (head * a.Q * a.G + rho) * a.NSB + (s0 >> a.sub_shift);
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
            if (blk && s0 + 16 * g < vis) {
              if (a.sub == 16) blk[g] = log2f(sum) + mx;
              else blk[g >> 1] = log2f(held = (g & 1 ? held : 0.f) + sum) + mx;
            }
          }
        }
        // ---- p = 2^(y - m + 11), sums by 16 slots
        const float off = m == -INFINITY ? 0.f : kPShift - m;
        float held = 0.f;
#pragma unroll
        for (int hh = 0; hh < 4; ++hh) {
          float pk[16];
#pragma unroll
          for (int g = 2 * hh; g < 2 * hh + 2; ++g) {
            const float4 t = tab[g];
            const float c = t.x * qscale, o = t.y + off;
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float p0 = fast_exp2(fmaf(s[16 * g + k], c, o)), p1 = fast_exp2(fmaf(s[16 * g + k + 1], c, o));
              s4[k & 2] += p0;
              s4[(k & 2) + 1] += p1;
              pk[(g & 1) * 8 + k / 2] = __uint_as_float(pack_h2(p0, p1));
            }
            const float sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
            if (!wild) {
              l = fmaf(sum, t.z, l);
              if (blk && s0 + 16 * g < vis) {
                if (a.sub == 16) blk[g] = log2f(sum) - (off + t.y);
                else blk[hh] = log2f(held = (g & 1 ? held : 0.f) + sum) - (off + t.y);
              }
            }
          }
          tmem_st16(tS + hh * 16, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[st]);
      }
      if (!ok) break;
      // ---- the item's rows, or this CTA's piece of them
      if (!wild) mx = m;
      float L = l, inv = 0.f;
      if (complete && live) {
        if (a.sink) L += fast_exp2(a.sink[hq] * kLog2e - mx);
        if (vis > 0) inv = 0x1p-11f / L * fast_exp2(m - mx);
        if (a.row_log) a.row_log[head * a.Q * a.G + rho] = log2f(L) + mx;
      }
      const int64_t slot = ((int64_t)blockIdx.x * 2 + (segment == 0 ? 0 : 1)) * kTcRows + st * 128 + row;
      if (!complete) a.part_ml[slot] = make_float4(m, mx, L, 0.f);
      if (count > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(&o_full[st], parity_o & 1, abort_sm))) break;
        ++parity_o;
        tc_fence_after();
      }
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + qrow * D;
      float* part = a.part_o + slot * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float v[32];
        if (count > 0) {
          tmem_ld32(tO + c, v);
          tmem_wait_ld();
        }
        if (!complete) {
#pragma unroll
          for (int k = 0; k < 32; k += 4) *reinterpret_cast<float4*>(part + c + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        } else if (live) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = vis > 0 ? v[k + 2 * i] * inv : 0.f, y = vis > 0 ? v[k + 2 * i + 1] * inv : 0.f;
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(x, y);
              w[i] = *reinterpret_cast<const uint32_t*>(&h2);
            }
            *reinterpret_cast<uint4*>(out + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      tc_fence_before();
      next_segment(u, count);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------- widen the codes --
    regs_dec<88>();
    constexpr int CH = D / 16;             // 16-byte chunks of a slot
    constexpr int PER = 128 / CH;          // slots a pass
    constexpr int NP = kTcTile / PER;      // passes
    const int t = tid & 127, c = t % CH, r0 = t / CH;
    const int flip = (c >> 2) & 1;         // which of a chunk's two fp16 chunks goes first: no bank conflicts
    uint4 kr[NP], vr[NP];
    Cursor pre = cur;
    long long up = u0;
    int64_t base = 0;   // code of the next tile's first slot
    int left = 0;       // slots of it that a query sees
    auto locate = [&]() {
      base = (((int64_t)((pre.e + e_base) / a.RT) * a.H + pre.h) * a.N + (int64_t)pre.local * kTcTile) * D;
      left = pre.n - pre.local * kTcTile;
    };
    auto load = [&](const uint8_t* codes, uint4 (&r)[NP]) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int slot = p * PER + r0;
        r[p] = slot < left ? ld_stream(codes + base + (int64_t)slot * D + c * 16) : make_uint4(0, 0, 0, 0);
      }
    };
    int at = 0;  // tiles written to the ring
    auto put = [&](const uint4 (&r)[NP]) -> bool {
      const int s = at % C::NS;
      if (!__all_sync(0xffffffffu, mbar_wait(&kv_empty[s], ((at / C::NS) & 1) ^ 1, abort_sm))) return false;
      uint8_t* dst = ring + s * C::row_tile + (c >> 2) * 16384;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int slot = p * PER + r0;
        uint4 w[2];
        widen4(r[p].x, w[0].x, w[0].y);
        widen4(r[p].y, w[0].z, w[0].w);
        widen4(r[p].z, w[1].x, w[1].y);
        widen4(r[p].w, w[1].z, w[1].w);
        uint8_t* line = dst + slot * 128;
        const int c0 = 2 * (c & 3);
        *reinterpret_cast<uint4*>(line + (((c0 + flip) ^ (slot & 7)) << 4)) = flip ? w[1] : w[0];
        *reinterpret_cast<uint4*>(line + (((c0 + 1 - flip) ^ (slot & 7)) << 4)) = flip ? w[0] : w[1];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kv_full[s]);
      ++at;
      return true;
    };
    if (pre.units > 0) {
      locate();
      load(a.kc, kr);
      while (up < u1) {
        load(a.vc, vr);
        if (!put(kr)) break;
        if (++up < u1) {
          pre.next(before, nmax, a.H, a.E);
          locate();
          load(a.kc, kr);
        }
        if (!put(vr)) break;
      }
    }
  } else {
    regs_dec<40>();
    if (warp == 12 && lane == 0) {
      // ------------------------------------------------------------- MMA --
      const uint32_t idesc_qk = idesc_f16(128, kTcTile), idesc_pv = idesc_f16(128, D, true);
      const uint32_t qb = smem_u32(sQ), rb = smem_u32(ring);
      int kv = 0, tiles = 0, segs = 0;  // ring tiles and tiles of each stream so far; segments with tiles
      bool ok = true;
      auto wait_kv = [&](int i) { return mbar_wait(&kv_full[i % C::NS], (i / C::NS) & 1, abort_sm); };
      auto issue_qk = [&](int s, int i) {  // S_s = Q_s K^T, K in ring tile i
        const uint32_t kb = rb + (i % C::NS) * C::row_tile;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_bf16(tbase + s * 128, sdesc_k_sw128(qb + s * C::row_tile + (k >> 2) * 16384 + (k & 3) * 32),
                   sdesc_k_sw128(kb + (k >> 2) * 16384 + (k & 3) * 32), idesc_qk, k > 0);
        mma_commit(&s_full[s]);
      };
      for (long long u = u0; ok && u < u1;) {
        const int count = segment_units(u);
        if (count > 0) {
          ok = wait_kv(kv);
          for (int s = 0; ok && s < 2; ++s) {
            ok = mbar_wait(&q_full[s], segs & 1, abort_sm);
            tc_fence_after();
            if (ok) issue_qk(s, kv);
          }
          if (ok) mma_commit(&kv_empty[kv % C::NS]);
          ++segs;
        }
        for (int i = 0; ok && i < count; ++i, ++tiles, kv += 2) {
          const uint32_t vb = rb + ((kv + 1) % C::NS) * C::row_tile;
          for (int s = 0; ok && s < 2; ++s) {
            if (s == 0) ok = wait_kv(kv + 1);
            ok = ok && mbar_wait(&p_full[s], tiles & 1, abort_sm);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kTcTile / 16; ++k)
              mma_f16_ts(tbase + 256 + s * D, tbase + s * 128 + k * 8, sdesc_mn_sw128(vb + k * 2048, 16384, 1024),
                         idesc_pv, i > 0 || k > 0);
            if (s == 1) mma_commit(&kv_empty[(kv + 1) % C::NS]);
            if (i + 1 < count) {
              if (s == 0) {
                ok = wait_kv(kv + 2);
                if (!ok) break;
                tc_fence_after();
              }
              issue_qk(s, kv + 2);
              if (s == 1) mma_commit(&kv_empty[(kv + 2) % C::NS]);
            } else {
              mma_commit(&o_full[s]);
            }
          }
        }
        next_segment(u, count);
      }
    }
    __syncwarp();
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
  if (warp == 12) tmem_dealloc(tbase, 512);
}

// Joins the pieces of the items that several CTAs share, a warp a row; rows of
// sequences without slots get their zeros here.
template <int D>
__global__ void __launch_bounds__(256) kv8_join(AttnArgs a, int launched) {
  pdl_wait();
  constexpr int parts = kTcRows / kJoinRows;
  const int64_t item = blockIdx.x / parts;
  const int e = (int)(item / a.H), h = (int)(item % a.H), b = e / a.RT, rt = e % a.RT;
  const int units = a.plan[e + 1] - a.plan[e], lane = threadIdx.x & 31;
  if (units > 0) {
    const Pieces pc(a, e, h, units, launched);
    if (pc.c0 == pc.c1) return;
  }
#pragma unroll 1
  for (int r = (int)(blockIdx.x % parts) * kJoinRows + (threadIdx.x >> 5), k = 0; k < kJoinRows / 8; r += 8, ++k) {
    const int64_t rho = (int64_t)rt * kTcRows + r;
    if (rho >= (int64_t)a.Q * a.G) return;
    const int j = (int)(rho / a.G), hq = h * a.G + (int)(rho % a.G);
    float v[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) v[i] = 0.f;
    if (units > 0) {
      const Pieces pc(a, e, h, units, launched);
      float M = -INFINITY, MX = -INFINITY, L = 0.f;
      for (int c = pc.c0; c <= pc.c1; ++c) {
        const float4 p = a.part_ml[pc.slot(c) * kTcRows + r];
        M = fmaxf(M, p.x);
        MX = fmaxf(MX, p.y);
      }
#pragma unroll 2
      for (int c = pc.c0; c <= pc.c1; ++c) {
        const int64_t sl = pc.slot(c) * kTcRows + r;
        const float4 p = a.part_ml[sl];
        const float f = p.x == -INFINITY ? 0.f : fast_exp2(p.x - M);
        L = fmaf(p.z, p.y == -INFINITY ? 0.f : fast_exp2(p.y - MX), L);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) v[i] = fmaf(a.part_o[sl * D + i * 32 + lane], f, v[i]);
      }
      if (a.sink) L += fast_exp2(a.sink[hq] * kLog2e - MX);
      if (a.row_log && lane == 0) a.row_log[((int64_t)b * a.H + h) * a.Q * a.G + rho] = log2f(L) + MX;
      const bool sees = a.n_vis[(int64_t)b * a.Q + j] > 0;
      const float inv = 0x1p-11f / L * fast_exp2(M - MX);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) v[i] = sees ? v[i] * inv : 0.f;
    }
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + (((int64_t)b * a.Q + j) * a.H * a.G + hq) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) out[i * 32 + lane] = __float2bfloat16_rn(v[i]);
  }
}

template <int D>
csa_status launch_tc(AttnArgs& a, cudaStream_t st) {
  auto kern = kv8_attend_tc_kernel<D>;
  const int smem = Tc<D>::total + 1024;
  if (!set_kernel_smem((const void*)kern, smem)) return CSA_ERR_CUDA;
  const long long items = (long long)a.E * a.H;
  a.planned = a.E <= kMaxPlan;
  long long grid = items;
  if (a.planned) {
    const long long units = items * ((a.N + kTcTile - 1) / kTcTile);
    grid = sm_count() < kMaxGrid ? sm_count() : kMaxGrid;
    if (units < grid) grid = units;
  }
  if (items * (kTcRows / kJoinRows) > 0x7fffffffll) return CSA_ERR_SHAPE;
  csa_status ok = CSA_OK;
  CSA_LAUNCH(KK_KV8_ATTEND, st,
             if (launch_maybe_pdl(true, kern, dim3((unsigned)grid), dim3(kTcThreads), smem, st, a) !=
                 cudaSuccess) ok = CSA_ERR_CUDA);
  if (a.planned)
    CSA_LAUNCH(KK_KV8_COMBINE, st,
               if (launch_maybe_pdl(true, kv8_join<D>, dim3((unsigned)(items * (kTcRows / kJoinRows))),
                                    dim3(256), 0, st, a, (int)grid) != cudaSuccess) ok = CSA_ERR_CUDA);
  return ok != CSA_OK ? ok : last_launch_status();
}

}  // namespace

bool kv8_attend_tc_takes(const csa_kv8_params& p, int B, int Q) {
  (void)B;
  return p.act == CSA_BF16 && p.d <= 128 && (int64_t)Q * (p.n_q / p.n_kv) > 128;
}
int kv8_attend_tc_rows() { return kTcRows; }

csa_status launch_kv8_attend_tc(const csa_kv8_params& p, AttnArgs& a, cudaStream_t st) {
  return p.d == 64 ? launch_tc<64>(a, st) : launch_tc<128>(a, st);
}

}  // namespace csa
