// kv8_attend.cu -- grouped-query attention over the 8-bit KV cache
// (csa_kv8_attend), the form for few query rows a KV head (decode).
//
// With x = scale log2(e) q . k (codes of the key times 2^ke) and y = x + ve
// (ve: the exponent of the value's block) the output is
//   sum_n 2^(y_n - M) c_n / sum_n 2^(y_n - ve_n - M),   M >= max y - 4,
// c_n the value's codes: E4M3 codes are exact in fp16, so both products run
// on codes as they are and every power of two goes into an exponent.  q is
// held as fp16 times a power of two per row (bf16 queries exactly; fp32 ones
// as two fp16 terms), p = 2^(y - M + 11) as one fp16 term or (fp32) two: the factor
// 2^11 uses fp16's range up to 2^15, so a term keeps 11 bits down to 2^-25 of the
// row's largest.  One term is off by 2^-11 of each weight at most, an eighth of bf16's
// half step; a second would cost every product of P V once more.
//
// What bounds it: the bytes of the cache, read once.  A CTA of 12 warps (d = 64:
// 16, d = 256: 6) works on one KV head and 16 query rows (heads of the group x
// queries); a unit is one tile of 32 slots per warp.  All units of the call lie on one line, cut
// into equal ranges, one per SM, so ragged lengths and any number of heads
// fill the machine evenly; the pieces of a head that ends up in several CTAs
// are joined by kv8_combine.  Each warp feeds itself: its lane 0 loads the
// tiles with TMA (128-byte swizzle: conflict-free fragment reads) into a ring
// of its own, and no barrier of the CTA is in the loop.  Both products are
// mma.sync m16n8k16: at 16 rows a head the loop needs about a third of that
// path's rate to keep up with HBM, and its operands come from registers, where
// the codes are widened, without a way through shared or tensor memory.
//
// 4 sequences of 1M tokens, 64 heads, 4 KV heads, d = 128: 709 to 766 us in long runs
// on different machines for 4.30 GB, 85 to 92% of the measured copy rate (638 in
// bursts, under the power limit); 32 of up to 64K tokens, 8 KV heads, with accumulated
// weights: 605 to 646 us for 3.26 GB, 77 to 82% (547 in bursts).  fp32 747 and 860.  With
// 8 warps 719 and 659 in bursts: a warp's 600 instructions a tile, not the loads, were
// waited for (issue slots 37% busy; 45% now).  One sequence of 1,111 tokens: 10 us
// in a graph, a chain of lengths (1.2), queries (1.6), 1.5 a unit, and the join
// of the warps (1.9).
#include <algorithm>

#include "kv8_attend.cuh"

namespace csa {

using namespace sm100;
using namespace kv8;

bool make_tmap_bf16(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols,
                    uint32_t box_rows);
bool tma_available();

namespace {

constexpr int kRows = 16;          // query rows of a CTA
constexpr int kTile = 32;          // slots of a warp's tile
constexpr int kJoinThreads = 256;
// A sequence of 2048 tokens, 2 KV heads (d = 128): one line 14.6 us, a CTA an item
// (6 units) 20.7; 17 sequences of 2496, 8 KV heads, fp32: 41.2 and 27.7.
constexpr int kJoinUnits = 4;
constexpr int kAccThreads = 256, kAccRows = 128, kAccFew = 32;
constexpr float kLazy = 4.f;       // the maximum may lag by 2^4: p <= 2^15 in fp16
constexpr float kPShift = 11.f;
// fp32: after so many tiles a warp adds O to a sum in tensor memory and starts anew.
// The tensor cores cut off what they add to an accumulator, towards zero: O of one
// sign shrank by 3.6e-8 a product, 5e-5 over 128K slots; in parts by less than 4e-6.
// It costs 1% (4 sequences of 1M, d = 128: 743 -> 747 us).  A sum in L2 cost 8%, every
// product added to O by itself 19%.  bf16, whose half step is 2^-8: after 512 tiles.
constexpr int kPart = 16, kPartBf16 = 512;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
template <int D, int SPLIT>
struct Cfg {
  static constexpr int NW = D == 64 ? 16 : D == 128 ? 12 : 6;  // warps
  static constexpr int threads = NW * 32;
  static constexpr int unit = NW * kTile;                // slots of a unit
  static constexpr int kv_bytes = kTile * D;             // one tile of K or V
  static constexpr int NS = D == 64 ? 3 : 2;             // tiles in a warp's ring
  static constexpr int warp_ring = NS * 2 * kv_bytes;    // (holds the warp's piece in the end: 16 rows of D + 4)
  static constexpr int steps = D / 16;
  // fp32: columns of tensor memory, D / 2 for a warp (four warps share the columns,
  // 32 lanes each)
  static constexpr int tmem_cols = D == 64 ? 128 : 256;
  // the last sum is taken up in the loop or (fp32, d = 128) by code behind it: fp32, 16
  // sequences of 64K, 4 KV heads, d = 256: 463 and 504 us; 4 of 1M, d = 128: 817 and 743;
  // bf16, 16 of 1M, 8 KV heads, d = 128: 5.63 and 5.72 ms
  static constexpr bool fold_last = SPLIT == 1 || D != 128;
  static constexpr int ring = 0;
  static constexpr int qfrag = ring + NW * warp_ring;
  static constexpr int ml = qfrag + SPLIT * steps * 32 * 16;
  static constexpr int rows = ml + NW * kRows * 16;      // per row: n_vis, exponent of q
  static constexpr int plan = rows + kRows * 8;          // units before, n_max: [E + 1], [E]
  static constexpr int bars = plan + (2 * kMaxPlan + 2) * 4;
  static constexpr int total = bars + NW * NS * 8 + 16;
  static_assert((NW + 3) / 4 * (D / 2) <= tmem_cols, "tensor memory");
  static_assert(kRows * (D + 4) * 4 <= warp_ring && total + 1024 <= 232448, "shared memory");
};

// WEIGHTS: a CTA has the only row tile of a sequence and KV head to the end, and adds
// its block weights up itself (a kernel of its own for it: the code would cost
// the long walk 1%)
// PARTS: a CTA may walk more than PT units of an item
template <typename T, int D, int SPLIT, bool WEIGHTS, bool PARTS>
__global__ void __launch_bounds__(Cfg<D, SPLIT>::threads, 1)
kv8_attend_mma(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               AttnArgs a) {
  using C = Cfg<D, SPLIT>;
  constexpr int PT = SPLIT == 2 ? kPart : kPartBf16;
  constexpr int NT = D / 8;  // output n-tiles
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = sm + C::ring;
  uint4* qfrag = reinterpret_cast<uint4*>(sm + C::qfrag);
  float4* ml = reinterpret_cast<float4*>(sm + C::ml);
  int2* rowinfo = reinterpret_cast<int2*>(sm + C::rows);
  int* before = reinterpret_cast<int*>(sm + C::plan);
  int* nmax = before + kMaxPlan + 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::bars);
  volatile int* abort_sm = reinterpret_cast<volatile int*>(bars + C::NW * C::NS);
  uint32_t* tmem_sm = reinterpret_cast<uint32_t*>(bars + C::NW * C::NS) + 1;
  __shared__ unsigned scan_sh[33];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (tid == 0) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    *abort_sm = 0;
    for (int i = 0; i < C::NW * C::NS; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
  }
  pdl_wait();
  if constexpr (!PARTS) pdl_trigger();
  long long u0, u1;
  int e_base;
  Cursor cur;
  if (!begin_line<C::threads>(a, kRows, C::unit, before, nmax, scan_sh, cur, u0, u1, e_base)) return;
  if constexpr (PARTS) {
    if (warp == 0) {
      tmem_alloc(tmem_sm, C::tmem_cols);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();  // (not before: a dependent that takes tensor memory first would wait for this CTA, and it for that)
  }
  int issued = 0, used = 0;  // tiles of this warp so far
  uint8_t* my_ring = ring + warp * C::warp_ring;
  uint64_t* my_bars = bars + warp * C::NS;
  const uint64_t policy = l2_evict_first_policy();

  long long u = u0;
  int segment = 0;
  while (u < u1) {
    // ---- a segment: the units of this range that belong to one item
    const int h = cur.h, b = (cur.e + e_base) / a.RT, rt = (cur.e + e_base) % a.RT;
    const int local0 = cur.local, units = cur.units;
    const int count = (int)min((long long)(units - local0), u1 - u);
    const int64_t head = (int64_t)b * a.H + h;
    fence_proxy_async_smem();  // the previous segment's piece in the ring, before loads go there
    __syncthreads();           // and its queries are free
    // ---- this warp's loads: of the segment only (the ring then holds its piece)
    const int first = (local0 * C::NW + warp) * kTile;  // slot of the warp's first tile
    const int tiles = cur.n > first ? min(count, (cur.n - first + C::unit - 1) / C::unit) : 0;
    const int64_t first_row = head * a.N + first;
    auto load = [&](int i) {
      if (i >= tiles) return;
      if (lane == 0) {
        const int st = issued % C::NS;
        const int row = (int)(D == 64 ? (first_row + (int64_t)i * C::unit) >> 1  // d = 64: two slots a 128-byte row
                                      : first_row + (int64_t)i * C::unit);
        uint8_t* dst = my_ring + st * 2 * C::kv_bytes;
        mbar_expect_tx(&my_bars[st], 2 * C::kv_bytes);
#pragma unroll
        for (int hf = 0; hf < (D == 256 ? 2 : 1); ++hf) {
          tma_load_2d_hint(dst + hf * kTile * 128, &tmK, &my_bars[st], hf * 64, row, policy);
          tma_load_2d_hint(dst + C::kv_bytes + hf * kTile * 128, &tmV, &my_bars[st], hf * 64, row, policy);
        }
      }
      ++issued;
    };
#pragma unroll 1
    for (int i = 0; i < C::NS; ++i) load(i);
    for (int r = warp; r < kRows; r += C::NW) {
      const int rho = rt * kRows + r, j = rho / a.G, hq = h * a.G + rho % a.G;
      const bool live = rho < a.Q * a.G;
      const int64_t qrow = (int64_t)b * a.Q + j;
      const T* q = reinterpret_cast<const T*>(a.q) + (qrow * a.H * a.G + hq) * D;
      float v[D / 32];
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        v[i] = live ? to_f32(q[i * 32 + lane]) : 0.f;
        const float f = fabsf(v[i]);
        amax = fmaxf(amax, f < INFINITY ? f : 0.f);
      }
      amax = warp_max(amax);
      // q * 2^-qe has its largest magnitude in [2^14, 2^15)
      const int qe = amax > 0.f ? (int)(__float_as_uint(amax) >> 23) - 127 - 14 : 0;
      const float f1 = pow2i(clamp_exp(-qe)), f2 = pow2i(-qe - clamp_exp(-qe));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int x = i * 32 + lane, xx = x % 128, c = xx / 16, y = xx % 16, z = y & 3;
        const int tt = D == 64 ? c : c >> 1;
        const int s = (D == 64 ? 0 : (x / 128) * 8 + (c & 1) * 4) + (y >> 2);
        const int idx = ((s * 32 + (r & 7) * 4 + tt) * 4 + (z >> 1) * 2 + (r >> 3)) * 2 + (z & 1);
        const float f = v[i] * f1 * f2;
        const __half hi = __float2half_rn(f);
        reinterpret_cast<__half*>(qfrag)[idx] = hi;
        if constexpr (SPLIT == 2)
          reinterpret_cast<__half*>(qfrag + C::steps * 32)[idx] = __float2half_rn(f - __half2float(hi));
      }
      if (lane == 0) rowinfo[r] = make_int2(live ? min(a.n_vis[qrow], a.N) : 0, qe);
    }
    __syncthreads();
    const int2 inf0 = rowinfo[g], inf1 = rowinfo[g + 8];
    const int vis[2] = {inf0.x, inf1.x}, qe[2] = {inf0.y, inf1.y};
    float m[2] = {-INFINITY, -INFINITY}, mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool wild = false;  // the sum relative to mx, the maximum of x
    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    // o += the sum in tensor memory (`begin`: there is none yet), under the present
    // reference; `away`: back there, and o starts anew
    float m_mem[2] = {-INFINITY, -INFINITY};
    auto add_part = [&](bool begin, bool away) {
      const uint32_t mem = *tmem_sm + ((uint32_t)((warp & 3) * 32) << 16) + (warp >> 2) * (D / 2);
      float f[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        f[r] = m_mem[r] == -INFINITY ? 0.f : fast_exp2(m_mem[r] - m[r]);
        m_mem[r] = m[r];
      }
      __syncwarp();
      tmem_wait_st();
#pragma unroll
      for (int n = 0; n < NT; n += 4) {
        float v[16];
        if (!begin) {
          tmem_ld16(mem + n * 4, v);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) o[n + k / 4][k % 4] = fmaf(v[k], f[k % 4 / 2], o[n + k / 4][k % 4]);
        }
        if (away) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            v[k] = o[n + k / 4][k % 4];
            o[n + k / 4][k % 4] = 0.f;
          }
          tmem_st16(mem + n * 4, v);
        }
      }
    };
    const uint8_t* ke_p = a.k_exp + head * a.NB;
    const uint8_t* ve_p = a.v_exp + head * a.NB;

#pragma unroll 1
    for (int i = 0; (PARTS && C::fold_last) || i < tiles; ++i) {
      if constexpr (PARTS)
        if (tiles > PT && i > 0 && (i % PT == 0 || i == tiles)) add_part(i == PT, i < tiles);
      if (PARTS && C::fold_last && i >= tiles) break;
      const int s0 = first + i * C::unit;
      // exponents of the tile's two halves (a tile may end beyond the cache)
      const int i0 = s0 >> a.shift, i1 = min((s0 + 16) >> a.shift, a.NB - 1);
      const int ke[2] = {(int)ke_p[i0] - 127, (int)ke_p[i1] - 127};
      const int ve[2] = {(int)ve_p[i0] - 127, (int)ve_p[i1] - 127};
      const int st = used % C::NS;
      if (!__all_sync(0xffffffffu, mbar_wait(&my_bars[st], (used / C::NS) & 1, abort_sm))) break;
      ++used;
      const uint8_t* ks = my_ring + st * 2 * C::kv_bytes;
      const uint8_t* vs = ks + C::kv_bytes;
      // ---- S = q K^T over codes
      float s[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[j][k] = 0.f;
#pragma unroll
      for (int hc = 0; hc < (D == 64 ? 1 : D / 64); ++hc) {  // 16-byte chunks of a slot's row
        uint4 kw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int tok = 8 * j + g;
          const uint8_t* p;
          if constexpr (D == 64)
            p = ks + (tok >> 1) * 128 + ((((tok & 1) * 4 + t) ^ ((tok >> 1) & 7)) << 4);
          else
            p = ks + (hc >> 1) * kTile * 128 + tok * 128 + (((2 * t + (hc & 1)) ^ (tok & 7)) << 4);
          kw[j] = *reinterpret_cast<const uint4*>(p);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint4 qa = qfrag[(hc * 4 + w) * 32 + lane];
          uint4 qb;
          if constexpr (SPLIT == 2) qb = qfrag[(C::steps + hc * 4 + w) * 32 + lane];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t b0, b1;
            widen4(w == 0 ? kw[j].x : w == 1 ? kw[j].y : w == 2 ? kw[j].z : kw[j].w, b0, b1);
            mma_f16(s[j], qa, b0, b1);
            if constexpr (SPLIT == 2) mma_f16(s[j], qb, b0, b1);
          }
        }
      }
      float tmax[2] = {-INFINITY, -INFINITY};
      const bool whole = __all_sync(0xffffffffu, min(vis[0], vis[1]) >= s0 + kTile);
      float half_sum[2][2];  // by half tile
      if (wild || max(abs(ve[0]), s0 + 16 < cur.n ? abs(ve[1]) : 0) > kTame) {
        if (!wild) {
          wild = true;
          mx[0] = m[0];
          mx[1] = m[1];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x[4][2], top = mx[r];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float c = a.scale2 * pow2i(clamp_exp(qe[r] + ke[j >> 1]));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              x[j][k] = s0 + 8 * j + 2 * t + k < vis[r] ? s[j][2 * r + k] * c : -INFINITY;
              top = fmaxf(top, x[j][k]);
            }
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          l[r] *= top > mx[r] ? fast_exp2(mx[r] - top) : 1.f;
          mx[r] = top;
          const float sub = top == -INFINITY ? 0.f : top;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            half_sum[r][hh] = (fast_exp2(x[2 * hh][0] - sub) + fast_exp2(x[2 * hh][1] - sub)) +
                              (fast_exp2(x[2 * hh + 1][0] - sub) + fast_exp2(x[2 * hh + 1][1] - sub));
            l[r] += half_sum[r][hh];
          }
        }
      }
      // ---- y = x + ve, running maximum
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float c = a.scale2 * pow2i(clamp_exp(qe[r] + ke[j >> 1]));
#pragma unroll
          for (int k = 0; k < 2; ++k) s[j][2 * r + k] = fmaf(s[j][2 * r + k], c, (float)ve[j >> 1]);
        }
      if (!whole) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (s0 + 8 * j + 2 * t + k >= vis[r]) s[j][2 * r + k] = -INFINITY;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) tmax[r] = fmaxf(tmax[r], fmaxf(s[j][2 * r], s[j][2 * r + 1]));
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        tmax[r] = fmaxf(tmax[r], __shfl_xor_sync(0xffffffffu, tmax[r], 1));
        tmax[r] = fmaxf(tmax[r], __shfl_xor_sync(0xffffffffu, tmax[r], 2));
      }
      if (__any_sync(0xffffffffu, tmax[0] > m[0] + kLazy || tmax[1] > m[1] + kLazy)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float m1 = fmaxf(m[r], tmax[r]);
          const float f = m1 > m[r] ? fast_exp2(m[r] - m1) : 1.f;
          m[r] = m1;
          if (!wild) l[r] *= f;
#pragma unroll
          for (int i2 = 0; i2 < NT; ++i2) {
            o[i2][2 * r] *= f;
            o[i2][2 * r + 1] *= f;
          }
        }
      }
      // ---- p = 2^(y - m + 11), its sums
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float sub = m[r] == -INFINITY ? 0.f : m[r] - kPShift;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float sum = 0.f;
#pragma unroll
          for (int j = 2 * hh; j < 2 * hh + 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              s[j][2 * r + k] = fast_exp2(s[j][2 * r + k] - sub);
              sum += s[j][2 * r + k];
            }
          if (!wild) {
            half_sum[r][hh] = sum;
            l[r] = fmaf(sum * 0x1p-11f, pow2i(clamp_exp(-ve[hh])), l[r]);
          }
        }
      }
      if (a.blk_log) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float h0 = half_sum[r][0], h1 = half_sum[r][1];
          h0 += __shfl_xor_sync(0xffffffffu, h0, 1);
          h1 += __shfl_xor_sync(0xffffffffu, h1, 1);
          h0 += __shfl_xor_sync(0xffffffffu, h0, 2);
          h1 += __shfl_xor_sync(0xffffffffu, h1, 2);
          const int rho = rt * kRows + g + 8 * r;
          if (t == 0 && vis[r] > s0) {
            float* dst = a.blk_log + (head * a.Q * a.G + rho) * a.NSB + (s0 >> a.sub_shift);
            const float base = m[r] - kPShift, b0 = wild ? mx[r] : base - ve[0], b1 = wild ? mx[r] : base - ve[1];
            if (a.sub == 32) {
              dst[0] = log2f(h0 + h1) + b0;
            } else {
              dst[0] = log2f(h0) + b0;
              if (vis[r] > s0 + 16) dst[1] = log2f(h1) + b1;
            }
          }
        }
        __syncwarp();
      }
      // ---- O += p V over codes; slots that no row sees may hold anything: the
      // item's last tile gets zeros there (whole slots, so swizzled rows too)
      const int lim = cur.n - s0;
      if (lim < kTile) {
        for (int i = lane; i < C::kv_bytes / 16; i += 32) {
          const int row = (i * 16 % (kTile * 128)) / 128;
          const int chunk = (i & 7) ^ (row & 7);  // where it stands before the swizzle
          const int tok = D == 64 ? 2 * row + (chunk >> 2) : row;
          if (tok >= lim) reinterpret_cast<uint4*>(my_ring + st * 2 * C::kv_bytes + C::kv_bytes)[i] = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint4 pa, pb;
        pa.x = pack_h2(s[2 * hh][0], s[2 * hh][1]);
        pa.y = pack_h2(s[2 * hh][2], s[2 * hh][3]);
        pa.z = pack_h2(s[2 * hh + 1][0], s[2 * hh + 1][1]);
        pa.w = pack_h2(s[2 * hh + 1][2], s[2 * hh + 1][3]);
        if constexpr (SPLIT == 2) {
          auto rest = [](uint32_t hi, float x, float y) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            return pack_h2(x - f.x, y - f.y);
          };
          pb.x = rest(pa.x, s[2 * hh][0], s[2 * hh][1]);
          pb.y = rest(pa.y, s[2 * hh][2], s[2 * hh][3]);
          pb.z = rest(pa.z, s[2 * hh + 1][0], s[2 * hh + 1][1]);
          pb.w = rest(pa.w, s[2 * hh + 1][2], s[2 * hh + 1][3]);
        }
        constexpr int VW = D == 64 ? 2 : 4;  // words of a slot's chunk
#pragma unroll
        for (int hf = 0; hf < (D == 256 ? 2 : 1); ++hf) {
          uint32_t vw[4][VW];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tok = 16 * hh + 2 * t + (k & 1) + (k >> 1) * 8;
            if constexpr (D == 64) {
              const int row = tok >> 1, ch = (tok & 1) * 4 + (g >> 1);
              const uint2 v2 = *reinterpret_cast<const uint2*>(vs + row * 128 + ((ch ^ (row & 7)) << 4) + (g & 1) * 8);
              vw[k][0] = v2.x;
              vw[k][1] = v2.y;
            } else {
              const uint4 v4 = *reinterpret_cast<const uint4*>(vs + hf * kTile * 128 + tok * 128 + ((g ^ (tok & 7)) << 4));
              vw[k][0] = v4.x;
              vw[k][1] = v4.y;
              vw[k][VW - 2] = v4.z;
              vw[k][VW - 1] = v4.w;
            }
          }
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            // pair the slots' bytes dim by dim: (slot 2t, slot 2t + 1) of dims 4w .. 4w + 3
            uint32_t b0[4], b1[4];
            widen4(__byte_perm(vw[0][w], vw[1][w], 0x5140), b0[0], b0[1]);
            widen4(__byte_perm(vw[0][w], vw[1][w], 0x7362), b0[2], b0[3]);
            widen4(__byte_perm(vw[2][w], vw[3][w], 0x5140), b1[0], b1[1]);
            widen4(__byte_perm(vw[2][w], vw[3][w], 0x7362), b1[2], b1[3]);
#pragma unroll
            for (int d4 = 0; d4 < 4; ++d4) {
              float(&acc)[4] = o[hf * 16 + w * 4 + d4];
              mma_f16(acc, pa, b0[d4], b1[d4]);
              if constexpr (SPLIT == 2) mma_f16(acc, pb, b0[d4], b1[d4]);
            }
          }
        }
      }
      if (lim < kTile) fence_proxy_async_smem();  // the zeros before a later load into the tile
      __syncwarp();  // the tile is read
      load(i + C::NS);
    }

    if constexpr (PARTS && !C::fold_last)
      if (tiles > PT) add_part(false, false);
    // ---- the warps' pieces become one
    u += max(count, 1);
    const bool complete = count == units;
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      float* dst = reinterpret_cast<float*>(my_ring) + (g + 8 * r) * (D + 4);
      if (t == 0) ml[warp * kRows + g + 8 * r] = make_float4(m[r], wild ? mx[r] : m[r], l[r], 0.f);
      // n-tile (hf, w): column 2t is dim 128 hf + (D == 64 ? 8 : 16) 2t + w
      constexpr int CH = D == 64 ? 8 : 16;
#pragma unroll
      for (int hf = 0; hf < (D == 256 ? 2 : 1); ++hf)
#pragma unroll
        for (int w = 0; w < CH; w += 4)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<float4*>(dst + hf * 128 + CH * (2 * t + k) + w) =
                make_float4(o[hf * CH + w][2 * r + k], o[hf * CH + w + 1][2 * r + k],
                            o[hf * CH + w + 2][2 * r + k], o[hf * CH + w + 3][2 * r + k]);
    }
    __syncthreads();
    {
      constexpr int TPR = C::threads / kRows;  // threads of a row
      const int r = tid / TPR, rho = rt * kRows + r;
      float M = -INFINITY, MX = -INFINITY, L = 0.f, f[C::NW];
#pragma unroll
      for (int w = 0; w < C::NW; ++w) {
        M = fmaxf(M, ml[w * kRows + r].x);
        MX = fmaxf(MX, ml[w * kRows + r].y);
      }
#pragma unroll
      for (int w = 0; w < C::NW; ++w) {
        const float4 v = ml[w * kRows + r];
        f[w] = v.x == -INFINITY ? 0.f : fast_exp2(v.x - M);
        L = fmaf(v.z, v.y == -INFINITY ? 0.f : fast_exp2(v.y - MX), L);
      }
      const bool live = rho < a.Q * a.G;
      float inv = 0.f, gap = 0.f;  // (their product may be below fp32's range where the output is not)
      const int j = rho / a.G, hq = h * a.G + rho % a.G;
      if (complete && live) {
        if (a.sink) L += fast_exp2(a.sink[hq] * kLog2e - MX);
        inv = 0x1p-11f / L;
        gap = fast_exp2(M - MX);
        if (a.row_log && tid % TPR == 0) a.row_log[head * a.Q * a.G + rho] = log2f(L) + MX;
      }
      const int64_t slot = (int64_t)blockIdx.x * 2 + (segment == 0 ? 0 : 1);
      if (!complete && tid % TPR == 0) a.part_ml[slot * kRows + r] = make_float4(M, MX, L, 0.f);
      T* out = reinterpret_cast<T*>(a.out) + (((int64_t)b * a.Q + j) * a.H * a.G + hq) * D;
      float* part = a.part_o + (slot * kRows + r) * D;
#pragma unroll 1
      for (int c = (tid % TPR) * 4; c < D; c += TPR * 4) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::NW; ++w) {
          const float4 v = *reinterpret_cast<const float4*>(ring + w * C::warp_ring + (r * (D + 4) + c) * 4);
          sum.x = fmaf(v.x, f[w], sum.x);
          sum.y = fmaf(v.y, f[w], sum.y);
          sum.z = fmaf(v.z, f[w], sum.z);
          sum.w = fmaf(v.w, f[w], sum.w);
        }
        if (!complete) {
          *reinterpret_cast<float4*>(part + c) = sum;
        } else if (live) {
          if (rowinfo[r].x <= 0) sum = make_float4(0.f, 0.f, 0.f, 0.f);
          else sum = make_float4(sum.x * inv * gap, sum.y * inv * gap, sum.z * inv * gap, sum.w * inv * gap);
          if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(out + c) = sum;
          } else {
            __nv_bfloat162 h2[2] = {__floats2bfloat162_rn(sum.x, sum.y), __floats2bfloat162_rn(sum.z, sum.w)};
            *reinterpret_cast<uint2*>(out + c) = *reinterpret_cast<uint2*>(h2);
          }
        }
      }
    }
    if constexpr (WEIGHTS) {
      __syncthreads();  // blk_log and row_log of the item's rows are this CTA's
      const int per = a.block / a.sub;
      for (int i = tid; i < a.NB; i += C::threads) {
        float sum = 0.f;
        bool seen = false;
        for (int r = 0; r < a.Q * a.G; ++r) {
          const int64_t lrow = head * a.Q * a.G + r;
          for (int k = 0; k < per; ++k)
            if ((i * per + k) * a.sub < rowinfo[r].x) {
              sum += fast_exp2(a.blk_log[lrow * a.NSB + i * per + k] - a.row_log[lrow]);
              seen = true;
            }
        }
        float* acc = a.acc + head * a.NB + i;
        if (seen) *acc = a.decay == 0.f ? sum : fmaf(a.decay, *acc, sum);
      }
    }
    ++segment;
    cur.local = local0 + count - 1;
    if (u < u1) cur.next(before, nmax, a.H, a.E);
    if (*abort_sm) break;
  }
  if (*abort_sm && lane == 0) {
    atomicOr(a.err, CSA_DEV_TIMEOUT);
    const uint64_t t0 = globaltimer();  // loads already issued land before the CTA leaves
    while (globaltimer() - t0 < 200000ull) __nanosleep(1000);
  }
  if constexpr (PARTS) {
    __syncwarp();
    tmem_wait_st();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(*tmem_sm, C::tmem_cols);
  }
}

// Joins the pieces of the heads that several CTAs share; one CTA a row, D / 4
// threads a piece, so that all pieces are under way at once.  Rows of sequences
// without slots get their zeros here.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) kv8_combine(AttnArgs a, int launched) {
  pdl_wait();
  const int r = (int)(blockIdx.x % kRows), tid = threadIdx.x;
  const int64_t item = blockIdx.x / kRows;
  const int e = (int)(item / a.H), h = (int)(item % a.H), b = e / a.RT, rt = e % a.RT;
  const int rho = rt * kRows + r;
  if (rho >= a.Q * a.G) return;
  const int j = rho / a.G, hq = h * a.G + rho % a.G;
  T* out = reinterpret_cast<T*>(a.out) + (((int64_t)b * a.Q + j) * a.H * a.G + hq) * D;
  const int units = a.plan[e + 1] - a.plan[e];
  if (units == 0) {
    for (int c = tid; c < D; c += kJoinThreads) out[c] = from_f32<T>(0.f);
    return;
  }
  const Pieces pc(a, e, h, units, launched);
  const int n = pc.c1 - pc.c0 + 1;  // at most kMaxGrid <= kJoinThreads
  if (n == 1) return;
  constexpr int per = D / 4, groups = kJoinThreads / per;
  __shared__ float red[32], red2[32], weight[kMaxGrid];
  __shared__ int64_t where[kMaxGrid];
  __shared__ float4 sums[groups][per];
  float4 ml = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
  if (tid < n) {
    where[tid] = pc.slot(pc.c0 + tid) * kRows + r;
    ml = a.part_ml[where[tid]];
  }
  const float M = block_reduce<true>(ml.x, red), MX = block_reduce<true>(ml.y, red2);
  if (tid < n) weight[tid] = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
  __syncthreads();  // (red is free again, too)
  float L = block_reduce<false>(ml.y == -INFINITY ? 0.f : ml.z * fast_exp2(ml.y - MX), red);
  const int g = tid / per, c4 = tid % per * 4;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = g; c < n; c += groups) {
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + where[c] * D + c4);
    const float f = weight[c];
    sum.x = fmaf(v.x, f, sum.x);
    sum.y = fmaf(v.y, f, sum.y);
    sum.z = fmaf(v.z, f, sum.z);
    sum.w = fmaf(v.w, f, sum.w);
  }
  sums[g][tid % per] = sum;
  __syncthreads();
  if (a.sink) L += fast_exp2(a.sink[hq] * kLog2e - MX);
  if (a.row_log && tid == 0) a.row_log[((int64_t)b * a.H + h) * a.Q * a.G + rho] = log2f(L) + MX;
  const bool sees = a.n_vis[(int64_t)b * a.Q + j] > 0;
  const float inv = 0x1p-11f / L, gap = fast_exp2(M - MX);
  for (int c = tid; c < D; c += kJoinThreads) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < groups; ++k) t += reinterpret_cast<const float*>(&sums[k][0])[c];
    out[c] = from_f32<T>(sees ? t * inv * gap : 0.f);
  }
}

// acc = decay acc + sum over the KV head's rows of the weight on a block, in a
// fixed order.  Few rows (decode): a warp sums 32 sub-blocks over all of them.
// Many: the 8 warps of a CTA share 32 sub-blocks, a row each at a time (128 bytes
// of blk_log), over at most kAccRows rows; the sums of several such parts go
// through the workspace (-1: no row sees the block) and kv8_acc_join adds them
// up.  blk_log is read once, which bounds it where there are many rows.
template <bool FEW>
__global__ void __launch_bounds__(kAccThreads) kv8_acc_kernel(AttnArgs a, int tiles, int parts, float* part) {
  pdl_wait();
  constexpr int W = kAccThreads / 32;
  __shared__ float red[W][33];
  const int tile = (int)(blockIdx.x % tiles), pt = (int)(blockIdx.x / tiles % parts);
  const int64_t head = blockIdx.x / tiles / parts;
  const int b = (int)(head / a.H), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sb = (FEW ? tile * W + warp : tile) * 32 + lane, slot = sb * a.sub;  // sub-block, its first slot
  const int rows = a.Q * a.G, r1 = min(rows, (pt + 1) * kAccRows);
  float sum = 0.f;
  bool seen = false;
#pragma unroll 4
  for (int r = pt * kAccRows + (FEW ? 0 : warp); r < r1; r += FEW ? 1 : W) {
    const int n = min(a.n_vis[(int64_t)b * a.Q + r / a.G], a.N);
    const int64_t lrow = head * rows + r;
    if (slot < n) {
      sum += fast_exp2(a.blk_log[lrow * a.NSB + sb] - a.row_log[lrow]);
      seen = true;
    }
  }
  if constexpr (!FEW) {
    red[warp][lane] = seen ? sum : -1.f;
    __syncthreads();
    if (warp > 0) return;
    sum = 0.f;
    seen = false;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float v = red[w][lane];
      seen |= v != -1.f;
      sum += v != -1.f ? v : 0.f;
    }
  }
  const int per = a.block / a.sub;  // 1, 2 or 4 lanes a block
  for (int o = 1; o < per; o <<= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    seen |= __shfl_xor_sync(0xffffffffu, (int)seen, o) != 0;
  }
  if (lane % per != 0 || sb >= a.NSB) return;
  const int64_t at = head * a.NB + sb / per;
  if (parts > 1)
    part[pt * ((int64_t)a.B * a.H * a.NB) + at] = seen ? sum : -1.f;
  else if (seen)
    a.acc[at] = a.decay == 0.f ? sum : fmaf(a.decay, a.acc[at], sum);
}
__global__ void __launch_bounds__(kAccThreads) kv8_acc_join(AttnArgs a, int parts, const float* part) {
  pdl_wait();
  const int64_t n = (int64_t)a.B * a.H * a.NB, at = (int64_t)blockIdx.x * kAccThreads + threadIdx.x;
  if (at >= n) return;
  float sum = 0.f;
  bool seen = false;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float v = part[p * n + at];
    seen |= v != -1.f;
    sum += v != -1.f ? v : 0.f;
  }
  if (seen) a.acc[at] = a.decay == 0.f ? sum : fmaf(a.decay, a.acc[at], sum);
}

// acc = decay acc for the blocks that some query of the sequence sees, before the
// parts of a call add to it one by one
__global__ void __launch_bounds__(kAccThreads) kv8_decay_kernel(AttnArgs a) {
  pdl_wait();
  __shared__ int red[kAccThreads / 32];
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  int n = 0;
  for (int j = threadIdx.x; j < a.Q; j += kAccThreads) n = max(n, min(a.n_vis[(int64_t)b * a.Q + j], a.N));
  n = __reduce_max_sync(0xffffffffu, n);
  if (lane == 0) red[threadIdx.x >> 5] = n;
  __syncthreads();
  n = __reduce_max_sync(0xffffffffu, lane < kAccThreads / 32 ? red[lane] : 0);
  const int i = blockIdx.x * kAccThreads + threadIdx.x;
  if (i >= a.NB || (int64_t)i * a.block >= n) return;
  for (int h = 0; h < a.H; ++h) {
    float* at = a.acc + ((int64_t)b * a.H + h) * a.NB + i;
    *at = a.decay == 0.f ? 0.f : a.decay * *at;
  }
}

struct Ws {
  size_t plan, part_ml, part_o, sum_o, row_log, acc_part, blk_log, total;
};

int mma_unit(const csa_kv8_params& p) {  // slots of a unit here
  return p.d == 64 ? Cfg<64, 1>::unit : p.d == 128 ? Cfg<128, 1>::unit : Cfg<256, 1>::unit;
}

// Which form the call takes: the one whose longest CTA is done first, at the time
// that a unit takes (measured on long prompts, tenths of a us; the tensor-core
// forms take 5 us more to set up).  64 heads, 8 of
// them KV heads, d = 128, bf16, here / two streams / one tile of 128 rows: 8
// sequences of 16K, 5 queries 144 us / 172 / 109, 16 queries 341 / 175 / -; 8 of
// 2K, 32 queries - / 64 / 48; one prompt of 32K, the last 2048 queries 11,400 / 2,150 /
// 2,580.
enum Form { kMma, kTc, kTc1 };
Form form_of(const csa_kv8_params& p, int B, int Q) {
  const bool f32 = p.act == CSA_F32;
  const long long rows = (long long)Q * (p.n_q / p.n_kv), heads = (long long)B * p.n_kv;
  auto cost = [&](int tile_rows, int unit, int join, int each) {
    return each * line_units((rows + tile_rows - 1) / tile_rows * heads, p.N, unit, kSms, join);
  };
  long long best = cost(kRows, mma_unit(p), kJoinUnits, f32 ? 31 : 24);
  Form form = kMma;
  if (rows <= 2 * kRows) return form;
  if (!f32 && p.d <= 128) {
    const long long c = 50 + cost(kv8_attend_tc_rows(), 128, kTcJoinUnits, 32);
    if (c < best) best = c, form = kTc;
  }
  const long long c = 50 + cost(kv8_attend_tc1_rows(), p.d == 256 ? 64 : 128, kTcJoinUnits,
                           p.d == 64 ? (f32 ? 21 : 19) : p.d == 128 ? (f32 ? 26 : 19) : (f32 ? 34 : 15));
  return c < best ? kTc1 : form;
}

struct Way {
  Form form;
  int rows;         // query rows of a CTA
  long long tiles;  // (sequence, row tile) pairs
  bool planned;     // the units of all items on one line
  bool parts;       // a CTA may walk so many slots of an item that O is summed up in parts
};
Way way_of(const csa_kv8_params& p, int B, int Q) {
  Way w;
  w.form = form_of(p, B, Q);
  w.rows = w.form == kTc ? kv8_attend_tc_rows() : w.form == kTc1 ? kv8_attend_tc1_rows() : kRows;
  w.tiles = ((long long)Q * (p.n_q / p.n_kv) + w.rows - 1) / w.rows * B;
  const int unit = w.form == kMma ? mma_unit(p) : w.form == kTc1 && p.d == 256 ? 64 : 128;
  const bool f32 = p.act == CSA_F32;
  const long long per = (p.N + (long long)unit - 1) / unit, items = w.tiles * p.n_kv;
  // of the tensor-core forms' bf16 sums, whose memory goes by CTA (share_of sees to it
  // that such calls fit a plan)
  const bool sums = w.form != kMma && !f32 && p.N > kPartSlots;
  // (the plan counts units in 32 bits)
  w.planned = w.tiles <= kMaxPlan && w.tiles * per <= 0x7fffffff &&
              (sums || on_a_line(items, p.N, unit, kSms, w.form == kMma ? kJoinUnits : kTcJoinUnits));
  const long long longest = w.planned ? std::min(per, items * per / kSms + 1) : per;
  w.parts = w.form == kMma ? longest > (f32 ? kPart : kPartBf16) : sums && w.planned && longest > kPartSlots / unit;
  return w;
}

int acc_parts(const csa_kv8_params& p, int Q) {
  return (int)(((long long)Q * (p.n_q / p.n_kv) + kAccRows - 1) / kAccRows);
}

Ws layout(const csa_kv8_params& p, int B, int Q, bool acc) {
  const Way way = way_of(p, B, Q);
  const size_t rows = (size_t)B * Q * p.n_q, pieces = way.planned ? (size_t)kMaxGrid * 2 * way.rows : 0;
  Ws w;
  w.plan = 0;
  w.part_ml = w.plan + (way.planned ? align_up((kMaxPlan + 1) * 4, 256) : 0);
  w.part_o = w.part_ml + pieces * 16;
  w.sum_o = w.part_o + pieces * p.d * 4;
  w.row_log = w.sum_o + (way.parts && way.form != kMma ? (size_t)kMaxGrid * way.rows * p.d * 4 : 0);
  w.acc_part = w.row_log + (acc ? align_up(rows * 4, 256) : 0);
  const int parts = acc_parts(p, Q);
  w.blk_log = w.acc_part + (acc && parts > 1 ? align_up((size_t)parts * B * p.n_kv * (p.N / p.block) * 4, 256) : 0);
  w.total = w.blk_log + (acc ? align_up(rows * (p.N / (p.block < 32 ? p.block : 32)) * 4, 256) : 0);
  return w;
}

// Accumulated weights go through a number per query row and sub-block (blk_log), 4
// bytes of workspace each: calls that would need more than this of them run as
// several, over as many sequences or, of one sequence, queries as fit.  512 MB are two
// milliseconds of attention (2048 queries of 64 heads over 32K slots: one call of 3.0
// ms; as two calls 3.1, so more of them cost 2 to 5%).
constexpr size_t kLogBytes = (size_t)512 << 20;
struct Share {
  int B, Q;  // sequences and queries of one call
};
Share log_share(const csa_kv8_params& p, int B, int Q, bool acc) {
  const size_t query = (size_t)p.n_q * (p.N / (p.block < 32 ? p.block : 32)) * 4, seq = query * Q;
  if (!acc || seq <= kLogBytes / B) return {B, Q};
  if (seq <= kLogBytes) {
    const long long most = (long long)(kLogBytes / seq), n = (B + most - 1) / most;
    return {(int)((B + n - 1) / n), Q};
  }
  const long long most = query < kLogBytes ? (long long)(kLogBytes / query) : 1, n = (Q + most - 1) / most;
  // whole tiles of 256 rows where that fits
  long long step = kv8_attend_tc_rows();
  for (int g = p.n_q / p.n_kv; g % 2 == 0 && step > 1; g /= 2) step /= 2;
  const long long even = (Q + n - 1) / n, full = (even + step - 1) / step * step;
  return {1, (int)(full <= most ? full : even)};
}

// bf16 prompts over so many slots that O is summed up in parts: those sums have memory
// for the CTAs of a plan, so row tiles that no plan holds go into calls of their own
// (of a tenth of a second and more).
Share share_of(const csa_kv8_params& p, int B, int Q, bool acc) {
  Share s = log_share(p, B, Q, acc);
  if (p.act == CSA_F32 || p.N <= kPartSlots || way_of(p, s.B, s.Q).form == kMma) return s;
  const long long rows = kv8_attend_tc1_rows(), G = p.n_q / p.n_kv;
  const long long most = std::min((long long)kMaxPlan, 0x7fffffffll / ((p.N + 63) / 64)), tiles = (s.Q * G + rows - 1) / rows;
  if (tiles <= most) s.B = (int)std::min((long long)s.B, most / tiles);
  else s.B = 1, s.Q = (int)std::max(1ll, most * rows / G);
  return s;
}

template <typename T, int D, int SPLIT>
csa_status launch_mma(const csa_kv8_params& p, const Kv8Cache& c, AttnArgs& a, bool weights, cudaStream_t st) {
  using C = Cfg<D, SPLIT>;
  CUtensorMap tmK, tmV;
  const uint64_t slots = (uint64_t)a.B * a.H * a.N;
  const uint64_t rows = D == 64 ? slots / 2 : slots, cols = D == 64 ? 64 : D / 2;
  const uint32_t box = D == 64 ? kTile / 2 : kTile;
  if (!make_tmap_bf16(&tmK, c.kc, rows, cols, box) || !make_tmap_bf16(&tmV, c.vc, rows, cols, box))
    return CSA_ERR_CUDA;
  auto kern = a.parts ? (weights ? kv8_attend_mma<T, D, SPLIT, true, true> : kv8_attend_mma<T, D, SPLIT, false, true>)
                      : (weights ? kv8_attend_mma<T, D, SPLIT, true, false> : kv8_attend_mma<T, D, SPLIT, false, false>);
  const int smem = C::total + 1024;
  if (!set_kernel_smem((const void*)kern, smem)) return CSA_ERR_CUDA;
  const long long items = (long long)a.E * a.H;
  long long grid = items;
  if (a.planned) {
    const long long units = items * ((a.N + C::unit - 1) / C::unit);
    grid = sm_count() < kMaxGrid ? sm_count() : kMaxGrid;
    if (units < grid) grid = units;
  }
  if (grid > 0x7fffffffll || items * kRows > 0x7fffffffll) return CSA_ERR_SHAPE;
  csa_status ok = CSA_OK;
  CSA_LAUNCH(KK_KV8_ATTEND, st,
             if (launch_maybe_pdl(true, kern, dim3((unsigned)grid), dim3(C::threads), smem, st, tmK,
                                  tmV, a) != cudaSuccess) ok = CSA_ERR_CUDA);
  if (a.planned)
    CSA_LAUNCH(KK_KV8_COMBINE, st,
               if (launch_maybe_pdl(true, kv8_combine<T, D>, dim3((unsigned)(items * kRows)),
                                    dim3(kJoinThreads), 0, st, a, (int)grid) != cudaSuccess) ok = CSA_ERR_CUDA);
  return ok != CSA_OK ? ok : last_launch_status();
}

csa_status attend(const csa_kv8_params& p, int B, int Q, float scale, const void* q, const int32_t* n_vis,
                  const Kv8Cache& c, const float* sink, void* out, float* acc, float decay, void* ws, cudaStream_t st) {
  AttnArgs a = {};
  a.q = q; a.n_vis = n_vis; a.kc = c.kc; a.vc = c.vc; a.k_exp = c.k_exp; a.v_exp = c.v_exp; a.sink = sink; a.out = out;
  a.B = B; a.Q = Q; a.H = p.n_kv; a.G = p.n_q / p.n_kv; a.N = p.N;
  a.NB = p.N / p.block; a.block = p.block;
  a.sub = p.block < 32 ? p.block : 32;
  a.NSB = p.N / a.sub;
  a.shift = 31 - __builtin_clz((unsigned)p.block);
  a.sub_shift = 31 - __builtin_clz((unsigned)a.sub);
  const Way way = way_of(p, B, Q);
  if (way.tiles > 0x7fffffffll) return CSA_ERR_SHAPE;
  a.E = (int)way.tiles;
  a.RT = a.E / B;
  a.planned = way.planned;
  a.parts = way.parts;
  const bool few = (long long)Q * a.G <= kAccFew;
  const int tiles = (a.NSB + (few ? kAccThreads : 32) - 1) / (few ? kAccThreads : 32), parts = acc_parts(p, Q);
  const long long blocks = (long long)B * a.H * a.NB;
  if ((long long)Q * a.G > 0x7fffffffll - kAccRows || (long long)B * a.H * tiles * parts > 0x7fffffffll ||
      blocks > 0x7fffffffll * kAccThreads)
    return CSA_ERR_SHAPE;
  a.scale2 = scale * kLog2e;
  a.decay = decay;
  a.err = device_error_word();
  if (a.err == nullptr) return CSA_ERR_CUDA;
  const Ws w = layout(p, B, Q, acc != nullptr);
  char* base = (char*)ws;
  a.plan = (int*)(base + w.plan);
  a.part_ml = (float4*)(base + w.part_ml);
  a.part_o = (float*)(base + w.part_o);
  a.sum_o = (float4*)(base + w.sum_o);
  if (acc) {
    a.acc = acc;
    a.row_log = (float*)(base + w.row_log);
    a.blk_log = (float*)(base + w.blk_log);
  }
  const bool weights = acc != nullptr && way.form == kMma && !way.planned && a.RT == 1;
  csa_status r;
  if (way.form == kTc)
    r = launch_kv8_attend_tc(p, a, st);
  else if (way.form == kTc1)
    r = launch_kv8_attend_tc1(p, a, st);
  else if (!tma_available())
    return CSA_ERR_CUDA;
  else if (p.act == CSA_F32)
    r = p.d == 64 ? launch_mma<float, 64, 2>(p, c, a, weights, st)
        : p.d == 128 ? launch_mma<float, 128, 2>(p, c, a, weights, st) : launch_mma<float, 256, 2>(p, c, a, weights, st);
  else
    r = p.d == 64 ? launch_mma<__nv_bfloat16, 64, 1>(p, c, a, weights, st)
        : p.d == 128 ? launch_mma<__nv_bfloat16, 128, 1>(p, c, a, weights, st)
                     : launch_mma<__nv_bfloat16, 256, 1>(p, c, a, weights, st);
  if (r != CSA_OK || !acc || weights) return r;
  float* part = (float*)(base + w.acc_part);
  csa_status ok = CSA_OK;
  CSA_LAUNCH(KK_KV8_ACC, st,
             if (launch_maybe_pdl(true, few ? kv8_acc_kernel<true> : kv8_acc_kernel<false>,
                                  dim3((unsigned)(B * a.H * tiles * parts)), dim3(kAccThreads), 0, st, a, tiles, parts,
                                  part) != cudaSuccess) ok = CSA_ERR_CUDA);
  if (parts > 1)
    CSA_LAUNCH(KK_KV8_ACC, st,
               if (launch_maybe_pdl(true, kv8_acc_join, dim3((unsigned)((blocks + kAccThreads - 1) / kAccThreads)),
                                    dim3(kAccThreads), 0, st, a, parts, (const float*)part) != cudaSuccess)
                 ok = CSA_ERR_CUDA);
  return ok != CSA_OK ? ok : last_launch_status();
}

}  // namespace

size_t kv8_attend_ws_bytes(const csa_kv8_params& p, int B, int Q, bool acc) {
  const Share s = share_of(p, B, Q, acc);
  size_t most = layout(p, s.B, s.Q, acc).total;
  if (B % s.B) most = std::max(most, layout(p, B % s.B, s.Q, acc).total);
  if (Q % s.Q) most = std::max(most, layout(p, s.B, Q % s.Q, acc).total);
  return most;
}

csa_status launch_kv8_attend(const csa_kv8_params& p, int B, int Q, float scale, const void* q,
                             const int32_t* n_vis, const Kv8Cache& c, const float* sink,
                             void* out, float* acc, float decay, void* ws, cudaStream_t st) {
  const Share s = share_of(p, B, Q, acc != nullptr);
  if (acc && s.Q < Q && decay != 1.f) {
    AttnArgs a = {};
    a.n_vis = n_vis; a.acc = acc; a.decay = decay;
    a.Q = Q; a.H = p.n_kv; a.N = p.N; a.NB = p.N / p.block; a.block = p.block;
    if (B > 65535) return CSA_ERR_SHAPE;
    csa_status ok = CSA_OK;
    CSA_LAUNCH(KK_KV8_ACC, st,
               if (launch_maybe_pdl(true, kv8_decay_kernel, dim3((unsigned)((a.NB + kAccThreads - 1) / kAccThreads), (unsigned)B),
                                    dim3(kAccThreads), 0, st, a) != cudaSuccess) ok = CSA_ERR_CUDA);
    if (ok != CSA_OK) return ok;
    decay = 1.f;
  }
  const int64_t row = (int64_t)p.n_q * p.d * (p.act == CSA_F32 ? 4 : 2), slots = (int64_t)p.n_kv * p.N,
                blocks = slots / p.block;
  for (int b = 0; b < B; b += s.B)
    for (int j = 0; j < Q; j += s.Q) {
      const int64_t r = (int64_t)b * Q + j;
      const csa_status ok = attend(
          p, std::min(s.B, B - b), std::min(s.Q, Q - j), scale, (const char*)q + r * row, n_vis + r,
          Kv8Cache{c.kc + b * slots * p.d, c.k_exp + b * blocks, c.vc + b * slots * p.d, c.v_exp + b * blocks}, sink,
          (char*)out + r * row, acc ? acc + b * blocks : nullptr, decay, ws, st);
      if (ok != CSA_OK) return ok;
    }
  return CSA_OK;
}

}  // namespace csa
