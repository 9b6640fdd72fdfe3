// kv8_evict.cu -- eviction of whole blocks from the 8-bit KV cache by their
// accumulated attention weight (csa_kv8_evict).
//
// kv8_select, one CTA per (sequence, KV head): a radix select over the
// order-preserving keys of acc finds the weight of the last block that stays;
// the blocks that stay become a bitmap in shared memory with a running count
// per word, from which every slot block reads off what it shall hold (the
// k-th free slot block takes the k-th kept block from keep-1 on).  It also
// moves what ends in slot block keep-1, whose own block may have to move
// first.  kv8_move copies the others: sources lie at keep or above and
// destinations below keep-1, so the copies are independent of one another.
//
// What bounds it: the bytes of the blocks that move, read and written once, and
// for short caches the chain of votes and scans of kv8_select.  8 sequences of
// 64K tokens cut to half (8 KV heads, d = 128, blocks of 64): 67 to 70 us for 361 MB,
// 79 to 82% of the measured copy rate (256 threads a block and one load of each cache
// in flight: 88 us; 64 threads 74, 8 loads 89).  A cache with few blocks beyond the
// budget is done in one kernel: 4 sequences, 125 blocks a head, one of them to go,
// 10.6 us as a graph of one call (12.7 with kv8_move behind it).
#include "common.cuh"
#include "kv8.h"

namespace csa {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 128;
constexpr int kFewMoves = 8;  // so many blocks a head are moved by kv8_select itself

struct EvictArgs {
  const float* acc;
  const int32_t* n_tok;
  Kv8Cache c;
  int32_t* kept;
  float* acc_out;
  int32_t* n_tok_out;
  unsigned* err;
  int H, N, NB, block, d, keep, recent;
  int alone;  // no kv8_move: at most kFewMoves blocks go, and n_tok_out is not n_tok
};

// NaN counts as the least weight; -0 + 0 is 0, so the two zeros tie
__device__ __forceinline__ uint32_t weight_key(float x) { return x == x ? score_key(x + 0.f) : 0u; }

// bits set below position i
__device__ __forceinline__ int rank_of(const uint32_t* bits, const int* before, int i) {
  return before[i >> 5] + __popc(bits[i >> 5] & ((1u << (i & 31)) - 1u));
}
// position of the k-th set bit (k from 0; it exists)
__device__ __forceinline__ int select_of(const uint32_t* bits, const int* before, int words, int k) {
  int lo = 0, hi = words;  // the last word with before[word] <= k
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= k) lo = mid; else hi = mid;
  }
  return lo * 32 + (int)__fns(bits[lo], 0, k - before[lo] + 1);
}

// running counts of set bits: before[w] = bits in words < w
__device__ void count_words(const uint32_t* bits, int* before, int words, unsigned* sh) {
  const int per = (words + kSelThreads - 1) / kSelThreads;
  const int w0 = min((int)threadIdx.x * per, words), w1 = min(w0 + per, words);
  unsigned n = 0, total;
  for (int w = w0; w < w1; ++w) n += __popc(bits[w]);
  unsigned at = block_exclusive_scan(n, sh, &total);
  for (int w = w0; w < w1; ++w) {
    before[w] = (int)at;
    at += __popc(bits[w]);
  }
  __syncthreads();
}

__device__ __forceinline__ void copy_block(const Kv8Cache& c, int64_t row, int NB, int block_bytes,
                                           int src, int dst, int tid, int threads) {
  const int n = block_bytes / 16;
  const uint4* ks = reinterpret_cast<const uint4*>(c.kc + (row * NB + src) * block_bytes);
  const uint4* vs = reinterpret_cast<const uint4*>(c.vc + (row * NB + src) * block_bytes);
  uint4* kd = reinterpret_cast<uint4*>(c.kc + (row * NB + dst) * block_bytes);
  uint4* vd = reinterpret_cast<uint4*>(c.vc + (row * NB + dst) * block_bytes);
  constexpr int U = 4;  // 16-byte loads of each cache in flight a thread (measured below)
  for (int i0 = tid; i0 < n; i0 += U * threads) {
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * threads < n) {
        a[u] = ks[i0 + u * threads];
        b[u] = vs[i0 + u * threads];
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * threads < n) {
        kd[i0 + u * threads] = a[u];
        vd[i0 + u * threads] = b[u];
      }
  }
  if (tid == 0) {
    c.k_exp[row * NB + dst] = c.k_exp[row * NB + src];
    c.v_exp[row * NB + dst] = c.v_exp[row * NB + src];
  }
}

__global__ void __launch_bounds__(kSelThreads) kv8_select_kernel(EvictArgs a) {
  extern __shared__ uint32_t sm[];
  const int words = (a.NB + 31) / 32;
  uint32_t* stay = sm;                                   // [words]
  int* before = reinterpret_cast<int*>(sm + words);      // [words]
  __shared__ unsigned sh[33];
  __shared__ unsigned hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_moves, moves[kFewMoves];
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int b = (int)(row / a.H), tid = threadIdx.x, lane = tid & 31;
  const int n = a.n_tok[b];
  const bool bad = n < 0 || n > a.N;
  if (bad && row % a.H == 0 && tid == 0) atomicOr(a.err, CSA_DEV_BAD_INDEX);
  const float* acc = a.acc + row * a.NB;
  float* acc_out = a.acc_out + row * a.NB;
  int32_t* kept = a.kept + row * a.keep;
  const int nb = bad ? 0 : (int)(((long long)n + a.block - 1) / a.block);
  if (a.alone && row % a.H == 0 && tid == 0) a.n_tok_out[b] = nb > a.keep ? n - (nb - a.keep) * a.block : n;
  if (nb <= a.keep) {  // nothing goes
    for (int i = tid; i < a.keep; i += kSelThreads) kept[i] = i < nb ? i : -1;
    for (int i = tid; i < a.NB; i += kSelThreads) {
      const float v = acc[i];
      acc_out[i] = i < nb || bad ? v : 0.f;
    }
    return;
  }
  const int cand = nb - a.recent;  // blocks that compete for the other places
  int need = a.keep - a.recent;
  uint32_t prefix = 0;
  int excess = 0;  // blocks whose key equals the last one's beyond the `need` that stay
  if (need > 0 && cand <= kSelThreads) {
    // one key a thread: the key of the need-th largest bit by bit, a vote of
    // the CTA each (32 votes take a microsecond, the passes below four)
    const uint32_t k = tid < cand ? weight_key(acc[tid]) : 0u;
    for (uint32_t bit = 0x80000000u; bit > 0; bit >>= 1)
      if (__syncthreads_count(tid < cand && k >= (prefix | bit)) >= need) prefix |= bit;
    need -= __syncthreads_count(tid < cand && k > prefix);
    excess = __syncthreads_count(tid < cand && k == prefix) - need;
  } else if (need > 0) {
    excess = 1;
    // the key of the need-th largest, 8 bits a pass
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int i = tid; i < cand; i += kSelThreads) {
        const uint32_t k = weight_key(acc[i]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1u);
      }
      __syncthreads();
      if (tid < 32) {  // from the top bucket down: lane l sums buckets 255-8l .. 248-8l
        unsigned sum = 0;
        for (int j = 0; j < 8; ++j) sum += hist[255 - 8 * lane - j];
        unsigned run = sum;
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned y = __shfl_up_sync(0xffffffffu, run, o);
          if (lane >= o) run += y;
        }
        const unsigned above = run - sum;
        if (above < (unsigned)need && run >= (unsigned)need) {
          unsigned at = above;
          int bkt = 255 - 8 * lane;
          while (at + hist[bkt] < (unsigned)need) at += hist[bkt--];
          s_prefix = prefix | ((uint32_t)bkt << shift);
          s_need = need - (int)at;
        }
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;  // places left among the keys that share the prefix
      __syncthreads();
    }
  }
  // blocks whose key equals the last one's: the first `need` of them stay
  if (excess > 0) {
    for (int i0 = (tid & ~31); i0 < words * 32; i0 += kSelThreads) {
      const int i = i0 + lane;
      const unsigned eq = __ballot_sync(0xffffffffu, i < cand && weight_key(acc[i]) == prefix);
      if (lane == 0) stay[i0 >> 5] = eq;
    }
    __syncthreads();
    count_words(stay, before, words, sh);
  }
  const bool choose = a.keep > a.recent;
  for (int i0 = (tid & ~31); i0 < words * 32; i0 += kSelThreads) {
    const int i = i0 + lane;
    bool s = i >= cand && i < nb;
    if (choose && i < cand) {
      const uint32_t k = weight_key(acc[i]);
      s = k > prefix || (k == prefix && (excess == 0 || rank_of(stay, before, i) < need));
    }
    const unsigned bits = __ballot_sync(0xffffffffu, s);
    __syncwarp();
    if (lane == 0) stay[i0 >> 5] = bits;
  }
  __syncthreads();
  count_words(stay, before, words, sh);
  if (tid == 0) s_moves = 0;
  __syncthreads();
  // what each slot block holds
  const int last = a.keep - 1;
  const int fixed = rank_of(stay, before, last);  // kept blocks that stay where they are
  for (int i = tid; i < a.keep; i += kSelThreads) {
    int src = nb - 1;
    if (i < last) {
      src = i;
      if (!((stay[i >> 5] >> (i & 31)) & 1u))
        src = select_of(stay, before, words, fixed + (i - rank_of(stay, before, i)));
    }
    kept[i] = src;
    if (i < last) acc_out[i] = acc[src];
    if (a.alone && i < last && src >= a.keep) moves[atomicAdd(&s_moves, 1)] = i;  // (their order does not matter)
  }
  // block keep-1, where it stays, goes to the first free slot block; then the
  // last block takes its place (the same thread moves the same bytes)
  const int block_bytes = a.block * a.d;
  if ((stay[last >> 5] >> (last & 31)) & 1u) {
    int free_slot = 0, hi = words;  // the first clear bit: the last word with all bits before it set
    while (hi - free_slot > 1) {
      const int mid = (free_slot + hi) >> 1;
      if (before[mid] == mid * 32) free_slot = mid; else hi = mid;
    }
    free_slot = free_slot * 32 + __ffs(~stay[free_slot]) - 1;
    copy_block(a.c, row, a.NB, block_bytes, last, free_slot, tid, kSelThreads);
  }
  copy_block(a.c, row, a.NB, block_bytes, nb - 1, last, tid, kSelThreads);
  const float acc_last = acc[nb - 1];
  __syncthreads();  // acc_out may be acc: all of it has been read
  if (tid == 0) acc_out[last] = acc_last;
  for (int i = a.keep + tid; i < a.NB; i += kSelThreads) acc_out[i] = 0.f;
  if (a.alone)  // (after the barrier: kept and the list are complete)
    for (int m = tid / kMoveThreads; m < s_moves; m += kSelThreads / kMoveThreads)
      copy_block(a.c, row, a.NB, block_bytes, kept[moves[m]], moves[m], tid % kMoveThreads, kMoveThreads);
}

__global__ void __launch_bounds__(kMoveThreads) kv8_move_kernel(EvictArgs a) {
  pdl_wait();
  const int64_t row = blockIdx.x / a.keep;
  const int i = (int)(blockIdx.x - row * a.keep);
  if (i == 0 && row % a.H == 0 && threadIdx.x == 0) {
    const int b = (int)(row / a.H), n = a.n_tok[b];
    const long long nb = ((long long)n + a.block - 1) / a.block;
    const bool over = n >= 0 && n <= a.N && nb > a.keep;
    a.n_tok_out[b] = over ? (int)(n - (nb - a.keep) * a.block) : n;
  }
  if (i >= a.keep - 1) return;
  const int src = a.kept[row * a.keep + i];
  if (src < a.keep) return;  // stays, holds nothing, or was moved with block keep-1
  copy_block(a.c, row, a.NB, a.block * a.d, src, i, threadIdx.x, kMoveThreads);
}

}  // namespace

csa_status launch_kv8_evict(const csa_kv8_params& p, int B, int keep, int recent,
                            const float* acc, const int32_t* n_tok, const Kv8Cache& c,
                            int32_t* kept, float* acc_out, int32_t* n_tok_out, cudaStream_t st) {
  EvictArgs a;
  a.acc = acc; a.n_tok = n_tok; a.c = c; a.kept = kept; a.acc_out = acc_out;
  a.n_tok_out = n_tok_out;
  a.err = device_error_word();
  if (a.err == nullptr) return CSA_ERR_CUDA;
  a.H = p.n_kv; a.N = p.N; a.NB = p.N / p.block; a.block = p.block; a.d = p.d;
  a.keep = keep; a.recent = recent;
  // a cache with a few blocks beyond the budget, as a decode loop keeps it: one
  // kernel (n_tok_out has to be other memory: all heads of a sequence read n_tok)
  a.alone = a.NB - keep <= kFewMoves && (n_tok_out + B <= n_tok || n_tok + B <= n_tok_out);
  const int smem = (a.NB + 31) / 32 * 8;
  if (smem > 40 * 1024 && !set_kernel_smem((const void*)kv8_select_kernel, smem)) return CSA_ERR_CUDA;
  const long long rows = (long long)B * p.n_kv;
  if (rows * keep > 0x7fffffffll) return CSA_ERR_SHAPE;
  csa_status ok = CSA_OK;
  CSA_LAUNCH(KK_KV8_SELECT, st,
             if (launch_maybe_pdl(true, kv8_select_kernel, dim3((unsigned)rows), dim3(kSelThreads), smem, st,
                                  a) != cudaSuccess) ok = CSA_ERR_CUDA);
  if (a.alone) return ok != CSA_OK ? ok : last_launch_status();
  CSA_LAUNCH(KK_KV8_MOVE, st,
             if (launch_maybe_pdl(true, kv8_move_kernel, dim3((unsigned)(rows * keep)),
                                  dim3(kMoveThreads), 0, st, a) != cudaSuccess) ok = CSA_ERR_CUDA);
  return ok != CSA_OK ? ok : last_launch_status();
}

}  // namespace csa
