// zf_sample_tokens: a token per row of logits by temperature, top-k, min-p and top-p, from given random numbers, and
// the distribution that is left.
//
//   w_i = exp((x_i - max) / temperature); candidates in the order of (x descending, i ascending): the first top_k,
//   of these the ones with w_i >= min_p, of these the shortest run from the front that has top_p of their sum;
//   the token is the first i (in index order) whose running sum of kept weights is above uniform * (their sum).
//
// All three filters keep a run from the front of that order, so together they are one threshold: a place
// (x, i), held as 64 bits that ascend along the order.  An entry's weight is an integer, exp2 to about 2^-31 of itself
// times 2^42, and sums of integers do not depend on how they are split, so neither does any choice that is made here;
// the choices agree with exact arithmetic but for borders within some 2^-30 of the point asked for.
//
// A cluster of up to 16 CTAs has a row, which is read from memory once and kept in shared memory (rows too large for
// that are read again from L2).  Passes over it, each ending in a cluster barrier:
//   1. the maximum;
//   2. (top-k, top-p) a histogram of the gap to the maximum, 4096 bins up to 24 temperatures.  It counts: a 32-bit
//      shared-memory atomic per entry, where sums of 64-bit weights would take several, and an exponential each.
//   3. (top-k) the bin with the k-th entry is exact; its entries are gathered into a list and ranked by comparing
//      each with each.
//   4. (top-p) counts times the bins' middle weights say in which bin the sum is reached; one pass sums the exact
//      weights before it and in it, and the neighbour is taken if the guess was wrong.  Its entries are listed and
//      ranked too.
//   5. sums of the kept weights per warp, then the piece, block and entry in which the drawn point lies;
//      probabilities are written along the way.
// A bin with more entries than the list holds is divided again by bits of the places, with exact sums.
//
// Bound: a row's bytes once from memory; the exponentials of steps 4 and 5 (about 30 instructions per entry that may
// be kept) and a chain of cluster barriers when there are few rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <climits>
#include <mutex>

#include "zf_device.cuh"
#include "zf_host.h"

namespace zf {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBins = 4096;
constexpr float kRange = 24.f;                     // temperatures that the bins cover
constexpr int kList = 1024;                        // entries that are ranked by comparing each with each
constexpr int kSub = 1024;                         // parts in which a crowded interval is divided

// 2^(j / 1024) in units of 2^-31, from repeated square roots of 2 (Newton's method in double).
struct Exp2Table {
  uint32_t v[1024];
};
constexpr double newton_sqrt(double x) {
  double r = x;
  for (int i = 0; i < 60; ++i) r = 0.5 * (r + x / r);
  return r;
}
constexpr Exp2Table make_exp2_table() {
  double root[10] = {};                            // 2^(1/2), 2^(1/4), .. 2^(1/1024)
  double r = 2.0;
  for (int k = 0; k < 10; ++k) {
    r = newton_sqrt(r);
    root[k] = r;
  }
  Exp2Table t{};
  for (int j = 0; j < 1024; ++j) {
    double p = 1.0;
    for (int k = 0; k < 10; ++k)
      if (j >> (9 - k) & 1) p *= root[k];
    t.v[j] = static_cast<uint32_t>(p * 2147483648.0 + 0.5);
  }
  return t;
}
__device__ const Exp2Table kExp2 = make_exp2_table();

struct SampleArgs {
  const void* logits;
  const float* uniform;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* probs;
  int32_t* status;
  long long row_stride;                            // entries
  int32_t rows, vocab;
  int32_t slice;                                   // entries per CTA (a multiple of 8)
  int32_t cached;                                  // whether a CTA keeps its slice in shared memory
  int32_t aligned;                                 // whether rows can be read 16 bytes at a time
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// A logit's place in the order of floats, ascending; NaN counts as -inf, -0 as +0.
__device__ __forceinline__ uint32_t order_of(float x) {
  x = x == x ? x + 0.f : -CUDART_INF_F;
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A row's exponential: x - max and its product with log2(e) / temperature are kept as pairs of floats.
struct Scale {
  float max, c_hi, c_lo, bins;                     // bins: bins per unit of x - max
};

struct Weight {
  uint32_t m;                                      // in [2^31, 2^32)
  int shift;                                       // the weight is m * 2^(shift - 31), shift <= 0
};
__device__ __forceinline__ Weight weight(const Scale& s, float x, const uint32_t* table) {
  // d = x - max exactly as d + e (Knuth's two-sum)
  const float d = __fadd_rn(x, -s.max);
  const float z = __fadd_rn(d, -x);
  const float e = __fadd_rn(__fadd_rn(x, -__fadd_rn(d, -z)), __fadd_rn(-s.max, -z));
  const float y = __fmul_rn(d, s.c_hi);
  const float l = __fmaf_rn(d, s.c_hi, -y) + __fmaf_rn(d, s.c_lo, e * s.c_hi);
  // y + l = k / 1024 + f, |f| <= 2^-11 and a little
  const float k = rintf(fmaxf(y, -4000.f) * 1024.f);
  const float f = __fmaf_rn(k, -0x1p-10f, fmaxf(y, -4000.f)) + l;
  const int j = static_cast<int>(k);
  // 2^f - 1 by its series, to 2^-36
  const float q = f * __fmaf_rn(f, __fmaf_rn(f, 0.0555041087f, 0.240226507f), 0.693147181f);
  const uint32_t t = table[j & 1023];
  const int m = static_cast<int>(t - 0x80000000u) + __float2int_rn(q * __uint2float_rn(t));
  // (k rounded up may leave m below 2^31 or above 2^32: the sum then moves a binade)
  Weight w;
  w.shift = j >> 10;
  const long long v = static_cast<long long>(m) + 0x80000000ll;
  if (v < 0x80000000ll) {
    w.m = static_cast<uint32_t>(v << 1);
    w.shift -= 1;
  } else if (v > 0xFFFFFFFFll) {
    w.m = static_cast<uint32_t>(v >> 1);
    w.shift += 1;
  } else {
    w.m = static_cast<uint32_t>(v);
  }
  return w;
}
__device__ __forceinline__ unsigned long long fixed(const Weight& w) {
  const int s = -w.shift;                          // 2^42 * m * 2^(shift - 31) = (m << 11) >> s
  const unsigned long long v = static_cast<unsigned long long>(w.m) << 11;
  if (s <= 0) return v << -s;
  return s > 43 ? 0ull : (v + (1ull << (s - 1))) >> s;
}
__device__ __forceinline__ float as_float(const Weight& w) {
  return w.shift < -126 ? 0.f : __uint2float_rn(w.m) * 0x1p-31f * __int_as_float((127 + w.shift) << 23);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(p)), "r"(rank));
  return addr;
}
__device__ __forceinline__ void remote_store(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long remote_load(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t remote_load32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t remote_add(uint32_t addr, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}
__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long x = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += x;
  }
  return v;
}

// ceil(p * n) for p in [0, 1], exactly.
__device__ __forceinline__ unsigned long long share_up(float p, unsigned long long n) {
  if (!(p > 0.f)) return 0;
  const uint32_t u = __float_as_uint(p);
  const int e = static_cast<int>(u >> 23) - 150;   // p = m * 2^e, m < 2^24
  if (e < -149) return n > 0;                      // (subnormal)
  const unsigned long long m = (u & 0x7FFFFFu) | 0x800000u;
  const unsigned long long lo = m * n, hi = __umul64hi(m, n);
  if (e >= 0) return n;
  const int s = -e;
  if (s >= 128) return n > 0;
  if (s >= 64) {
    const unsigned long long q = s == 64 ? hi : hi >> (s - 64);
    const bool rest = lo != 0 || (s > 64 && (hi << (128 - s)) != 0);
    return q + rest;
  }
  const unsigned long long q = (hi << (64 - s)) | (lo >> s);
  return q + ((lo << (64 - s)) != 0);
}
// floor(p * n).
__device__ __forceinline__ unsigned long long share_down(float p, unsigned long long n) {
  const unsigned long long up = share_up(p, n);
  if (up == 0) return 0;
  // up is exact when up * 2^s equals m * n; the next lower integer otherwise
  const uint32_t u = __float_as_uint(p);
  const int e = static_cast<int>(u >> 23) - 150;
  if (e < -149) return 0;
  if (e >= 0) return n;
  const unsigned long long m = (u & 0x7FFFFFu) | 0x800000u;
  const unsigned long long lo = m * n, hi = __umul64hi(m, n);
  const int s = -e;
  if (s >= 128) return 0;
  if (s >= 64) return s == 64 ? hi : hi >> (s - 64);
  return (hi << (64 - s)) | (lo >> s);
}

struct Entry {
  unsigned long long at, w;                        // place, weight or 1
};

// What the CTAs of a cluster exchange and share.
struct Shared {
  unsigned long long sums[kMaxCluster * kWarps];   // of every warp of the cluster (pushed to all CTAs)
  unsigned long long part[2][kMaxCluster][3];      // per CTA, alternating: sums of a pass
  Entry list[kList];                               // (CTA 0's is the cluster's)
  uint32_t listed;                                 // entries in it
  uint32_t bins[kBins];                            // counts; the cluster's sums in every CTA after fold()
  unsigned long long sub[kSub];                    // weights of the parts of an interval
  uint32_t table[1024];
  unsigned long long red[kWarps];
  unsigned long long out[4];                       // a threshold and sums found by one thread, for all CTAs
};

template <typename T, bool kVec>
struct Row {
  const T* at;                                     // this CTA's slice
  int first, n;                                    // index of its first entry, entries
};

// f(index, x) for every entry of the CTA's slice.  kVec: 16 bytes at a time (the slice starts on 16 bytes and may be
// read to a multiple of them).
template <typename T, bool kVec, typename F>
__device__ __forceinline__ void for_row(const Row<T, kVec>& r, F&& f) {
  if (kVec) {
    constexpr int kPer = 16 / sizeof(T);
    for (int i = threadIdx.x * kPer; i < r.n; i += kThreads * kPer) {
      T v[kPer];
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(r.at + i);
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (i + e < r.n) f(r.first + i + e, to_float(v[e]));
    }
  } else {
    for (int i = threadIdx.x; i < r.n; i += kThreads) f(r.first + i, to_float(r.at[i]));
  }
}

// A place in the order: (max - x, index).
__device__ __forceinline__ unsigned long long place(uint32_t top, float x, int i) {
  return (static_cast<unsigned long long>(top - order_of(x)) << 32) | static_cast<uint32_t>(i);
}
__device__ __forceinline__ int bin_of(const Scale& s, float x) {
  const float g = (s.max - x) * s.bins;            // (NaN: a NaN logit, in the last bin)
  return g < static_cast<float>(kBins - 1) ? static_cast<int>(g) : kBins - 1;
}

struct Ctx {
  Shared* sh;
  uint32_t rank, ranks;
  int flip;                                        // which part[] the next exchange uses
};

// Block sums of three values, then sums over the cluster (every thread gets them).
__device__ __forceinline__ void cluster_sums(Ctx& c, unsigned long long (&v)[3]) {
  Shared& sh = *c.sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ unsigned long long red[3][kWarps];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const unsigned long long s = warp_sum(v[k]);
    if (lane == 0) red[k][warp] = s;
  }
  __syncthreads();
  if (warp < 3) {
    const unsigned long long s = warp_sum(lane < kWarps ? red[warp][lane] : 0);
    if (lane < static_cast<int>(c.ranks)) remote_store(remote(&sh.part[c.flip][c.rank][warp], lane), s);
  }
  cluster_sync();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    v[k] = 0;
    for (uint32_t r = 0; r < c.ranks; ++r) v[k] += sh.part[c.flip][r][k];
  }
  c.flip ^= 1;
  __syncthreads();                                 // (red is free again)
}

__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, unsigned long long* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_sum(v);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return warp_sum(lane < kWarps ? red[lane] : 0);
}

// The cluster's sums of bins[0 .. n) into every CTA's bins.
__device__ __forceinline__ void fold_bins(Ctx& c, uint32_t* bins, int n) {
  if (c.ranks == 1) {
    __syncthreads();
    return;
  }
  cluster_sync();
  const int per = (n + static_cast<int>(c.ranks) - 1) / static_cast<int>(c.ranks);
  const int lo = static_cast<int>(c.rank) * per, hi = min(n, lo + per);
  for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
    uint32_t s = 0;
    for (uint32_t r = 0; r < c.ranks; ++r) s += remote_load32(remote(&bins[i], r));
    for (uint32_t r = 0; r < c.ranks; ++r)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(&bins[i], r)), "r"(s) : "memory");
  }
  cluster_sync();
}
__device__ __forceinline__ void fold_sub(Ctx& c, unsigned long long* sub, int n) {
  if (c.ranks == 1) {
    __syncthreads();
    return;
  }
  cluster_sync();
  const int per = (n + static_cast<int>(c.ranks) - 1) / static_cast<int>(c.ranks);
  const int lo = static_cast<int>(c.rank) * per, hi = min(n, lo + per);
  for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
    unsigned long long s = 0;
    for (uint32_t r = 0; r < c.ranks; ++r) s += remote_load(remote(&sub[i], r));
    for (uint32_t r = 0; r < c.ranks; ++r) remote_store(remote(&sub[i], r), s);
  }
  cluster_sync();
}

// The first of n values whose running sum reaches target (>= 1), and the sum before it, in every thread.  n a multiple
// of kThreads.  -1 when the total stays below.
template <typename Value>
__device__ __forceinline__ int reach(int n, unsigned long long target, unsigned long long& before, Value&& value) {
  __shared__ unsigned long long red[kWarps];
  __shared__ int found;
  __shared__ unsigned long long found_before;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = n / kThreads;
  unsigned long long own = 0;
  for (int k = 0; k < per; ++k) own += value(threadIdx.x * per + k);
  const unsigned long long in = warp_scan(own, lane);
  if (lane == 31) red[warp] = in;
  if (threadIdx.x == 0) found = -1;
  __syncthreads();
  unsigned long long base = 0;
  for (int w = 0; w < warp; ++w) base += red[w];
  unsigned long long at = base + in - own;
  if (at < target && at + own >= target) {         // one thread at most
    for (int k = 0; k < per; ++k) {
      const unsigned long long v = value(threadIdx.x * per + k);
      if (at + v >= target) {
        found = threadIdx.x * per + k;
        found_before = at;
        break;
      }
      at += v;
    }
  }
  __syncthreads();
  const int f = found;
  before = found_before;
  __syncthreads();
  return f;
}

// Among the listed entries: the place at which the running sum along the order reaches target (>= 1), and that sum
// without it.  CTA 0 finds it, all get it.
__device__ __forceinline__ unsigned long long rank_list(Ctx& c, unsigned long long target, unsigned long long& before) {
  Shared& sh = *c.sh;
  cluster_sync();                                  // the list is complete
  if (c.rank == 0) {
    const int n = min(sh.listed, static_cast<uint32_t>(kList));
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const Entry own = sh.list[i];
      unsigned long long sum = 0;
      for (int j = 0; j < n; ++j) {
        const Entry o = sh.list[j];
        if (o.at <= own.at) sum += o.w;
      }
      if (sum >= target && sum - own.w < target)
        for (uint32_t r = 0; r < c.ranks; ++r) {
          remote_store(remote(&sh.out[0], r), own.at);
          remote_store(remote(&sh.out[1], r), sum - own.w);
        }
    }
  }
  cluster_sync();
  before = sh.out[1];
  return sh.out[0];
}

__device__ __forceinline__ void append(Ctx& c, unsigned long long at, unsigned long long w) {
  const uint32_t k = remote_add(remote(&c.sh->listed, 0), 1);
  if (k < kList) {
    const uint32_t to = remote(&c.sh->list[k], 0);
    remote_store(to, at);
    remote_store(to + 8, w);
  }
}
__device__ __forceinline__ void clear_list(Ctx& c) {
  if (threadIdx.x == 0) {
    c.sh->listed = 0;
    c.sh->out[0] = ~0ull;                          // (a sum that is not reached keeps all)
    c.sh->out[1] = 0;
  }
  cluster_sync();
}

// The place at which the running sum of value(i, x) (1 or a weight; entries that are not in are skipped) along the order
// reaches target, where it is known to lie in bin b, before which the sum is `before` (updated to the sum before the
// place).  n: an upper bound of the entries in the bin.
template <typename T, bool kVec, typename In, typename Val>
__device__ __forceinline__ unsigned long long settle(Ctx& c, const Row<T, kVec>& row, const Scale& s, uint32_t top, int b,
                                                     uint32_t n, unsigned long long target, unsigned long long& before,
                                                     In&& in, Val&& value) {
  Shared& sh = *c.sh;
  unsigned long long lo = 0, hi = ~0ull;           // places
  if (n > kList) {
    // the interval's ends, then parts of it by their bits
    unsigned long long mn = ~0ull, mx = 0;
    for_row(row, [&](int i, float x) {
      if (bin_of(s, x) == b && in(i, x)) {
        const unsigned long long p = place(top, x, i);
        mn = min(mn, p);
        mx = max(mx, p);
      }
    });
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      mn = min(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, d));
      mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    }
    const int me = static_cast<int>(c.rank) * kWarps + (threadIdx.x >> 5);
    for (int pass = 0; pass < 2; ++pass) {
      cluster_sync();
      if ((threadIdx.x & 31) < c.ranks) remote_store(remote(&sh.sums[me], threadIdx.x & 31), pass ? mx : mn);
      cluster_sync();
      for (uint32_t k = 0; k < c.ranks * kWarps; ++k) {
        const unsigned long long v = sh.sums[k];
        if (pass) hi = k ? max(hi, v) : v;
        else lo = k ? min(lo, v) : v;
      }
    }
    while (n > kList && lo < hi) {
      int shift = 0;
      while (((hi - lo) >> shift) >= kSub) ++shift;
      cluster_sync();
      for (int k = threadIdx.x; k < kSub; k += kThreads) {
        sh.sub[k] = 0;
        sh.bins[k] = 0;
      }
      __syncthreads();
      for_row(row, [&](int i, float x) {
        if (bin_of(s, x) != b || !in(i, x)) return;
        const unsigned long long p = place(top, x, i);
        if (p < lo || p > hi) return;
        const int k = static_cast<int>((p - lo) >> shift);
        atomicAdd(&sh.bins[k], 1u);
        atomicAdd(&sh.sub[k], value(x));
      });
      __syncthreads();
      fold_bins(c, sh.bins, kSub);
      fold_sub(c, sh.sub, kSub);
      unsigned long long inner;
      int k = reach(kSub, target - before, inner, [&](int j) { return sh.sub[j]; });
      if (k < 0) {                                 // (not reached: the target lies within)
        k = kSub - 1;
        inner = 0;
      }
      before += inner;
      n = sh.bins[k];
      lo += static_cast<unsigned long long>(k) << shift;
      hi = min(hi, lo + ((1ull << shift) - 1));
    }
    if (lo >= hi) return lo;
  }
  clear_list(c);
  for_row(row, [&](int i, float x) {
    if (bin_of(s, x) != b || !in(i, x)) return;
    const unsigned long long p = place(top, x, i);
    if (p >= lo && p <= hi) append(c, p, value(x));
  });
  unsigned long long inner;
  const unsigned long long at = rank_list(c, target - before, inner);
  before += inner;
  return at;
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  T* cache = reinterpret_cast<T*>(raw + ((sizeof(Shared) + 15) & ~static_cast<size_t>(15)));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Ctx c{&sh, cluster_rank(), cluster_size(), 0};
  const int r = blockIdx.x / c.ranks, V = a.vocab;
  for (int k = tid; k < 1024; k += kThreads) sh.table[k] = kExp2.v[k];
  allow_next_grid();
  wait_prior_grid();
  cluster_sync();                                  // all CTAs run before their shared memory is written

  // ---- the row, and its maximum
  Row<T, kVec> row;
  row.first = min(V, static_cast<int>(c.rank) * a.slice);
  row.n = min(V - row.first, a.slice);
  row.at = static_cast<const T*>(a.logits) + static_cast<long long>(r) * a.row_stride + row.first;
  uint32_t most = 0;
  if (a.cached) {
    if (a.aligned) {
      constexpr int kPer = 16 / sizeof(T);
      constexpr int kDeep = 4;
      for (int i0 = tid * kPer; i0 < row.n; i0 += kThreads * kPer * kDeep) {
        uint4 v[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
          const int i = i0 + k * kThreads * kPer;
          if (i < row.n) v[k] = *reinterpret_cast<const uint4*>(row.at + i);
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
          const int i = i0 + k * kThreads * kPer;
          if (i < row.n) *reinterpret_cast<uint4*>(cache + i) = v[k];
        }
      }
    } else {
#pragma unroll 8
      for (int i = tid; i < row.n; i += kThreads) cache[i] = row.at[i];
    }
    row.at = cache;
    __syncthreads();
  }
  for_row(row, [&](int, float x) { most = max(most, order_of(x)); });
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane < static_cast<int>(c.ranks)) remote_store(remote(&sh.sums[c.rank * kWarps + warp], lane), most);
  cluster_sync();
  uint32_t top = 0;
  for (int k = lane; k < static_cast<int>(c.ranks) * kWarps; k += 32) top = max(top, static_cast<uint32_t>(sh.sums[k]));
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  const uint32_t bits = top & 0x80000000u ? top & 0x7FFFFFFFu : ~top;
  Scale s;
  s.max = __uint_as_float(bits);

  // ---- the row's parameters
  const float temp = a.temperature ? a.temperature[r] : 1.f;
  int k_top = a.top_k ? a.top_k[r] : 0;
  const float p_top = a.top_p ? a.top_p[r] : 1.f, p_min = a.min_p ? a.min_p[r] : 0.f;
  const float u = a.uniform ? a.uniform[r] : 0.f;
  const bool bad = !(fabsf(s.max) < CUDART_INF_F) || !(temp >= 0.f && temp < CUDART_INF_F) || k_top < 0 || !(p_top >= 0.f) ||
                   !(p_min <= 1.f) || !(u >= 0.f && u < 1.f);
  if (bad) {                                       // the whole cluster
    if (c.rank == 0 && tid == 0) {
      report(a.status, ZF_DEV_BAD_PROBS);
      if (a.tokens) a.tokens[r] = -1;
    }
    if (a.probs)
      for (int i = tid; i < row.n; i += kThreads) a.probs[static_cast<size_t>(r) * V + row.first + i] = 0.f;
    return;
  }
  const bool greedy = temp < 1e-6f;                // (the largest logit, the first of equal ones)
  if (greedy) k_top = 1;
  const double inv = 1.4426950408889634 / (greedy ? 1.0 : static_cast<double>(temp));
  s.c_hi = static_cast<float>(inv);
  s.c_lo = static_cast<float>(inv - static_cast<double>(s.c_hi));
  s.bins = static_cast<float>(kBins) / (kRange * (greedy ? 1.f : temp));
  auto exact = [&](float x) { return fixed(weight(s, x, sh.table)); };

  unsigned long long limit = ~0ull;                // the last place that is kept
  const bool by_k = k_top > 0 && k_top < V, by_p = p_top < 1.f && !greedy, by_min = p_min > 0.f;
  if (by_k || by_p) {
    for (int k = tid; k < kBins; k += kThreads) sh.bins[k] = 0;
    __syncthreads();
    for_row(row, [&](int, float x) { atomicAdd(&sh.bins[bin_of(s, x)], 1u); });
    __syncthreads();
    fold_bins(c, sh.bins, kBins);
  }
  int b_k = kBins - 1;                             // the bin with the k-th entry
  uint32_t n_k = 0;
  unsigned long long before_k = 0;
  if (by_k) {
    b_k = reach(kBins, static_cast<unsigned long long>(k_top), before_k, [&](int j) { return sh.bins[j]; });
    n_k = sh.bins[b_k];
  }
  // smallest weight that min-p keeps: compared as m * 2^(shift - 31)
  auto above_min = [&](float x) {
    if (!by_min) return true;
    const Weight w = weight(s, x, sh.table);
    const float f = as_float(w);
    if (f > p_min * 1.000001f) return true;
    if (f < p_min * 0.999999f) return false;
    // close: in 32 bits of fraction
    int e;
    const float m = frexpf(p_min, &e);             // p_min = m 2^e, m in [0.5, 1)
    const unsigned long long want = static_cast<unsigned long long>(m * 16777216.f) << 8;   // m 2^32
    const int d = w.shift + 1 - e;                 // w = (m_w / 2^32) 2^(shift + 1)
    return d == 0 ? static_cast<unsigned long long>(w.m) >= want : d > 0;
  };
  if (by_k) {
    // settle() overwrites the bins when it divides: what top-p needs of them is kept only if it does not
    limit = settle(c, row, s, top, b_k, n_k, static_cast<unsigned long long>(k_top), before_k,
                   [&](int, float) { return true; }, [](float) { return 1ull; });
  }
  auto kept = [&](int i, float x) { return place(top, x, i) <= limit && above_min(x); };
  if (by_p) {
    if (by_k && n_k > kList) {                     // the counts again
      cluster_sync();
      for (int k = tid; k < kBins; k += kThreads) sh.bins[k] = 0;
      __syncthreads();
      for_row(row, [&](int, float x) { atomicAdd(&sh.bins[bin_of(s, x)], 1u); });
      __syncthreads();
      fold_bins(c, sh.bins, kBins);
    }
    // middle weights of the bins in units of 2^-20, the last bin's and those that min-p drops without any
    const int b_min = by_min ? bin_of(s, s.max + log2f(p_min) / s.c_hi) : kBins - 1;
    auto guess = [&](int j) -> unsigned long long {
      if (j > b_k || j > b_min || j == kBins - 1) return 0;
      const uint32_t n = j == b_k && by_k ? static_cast<uint32_t>(k_top - before_k) : sh.bins[j];
      return static_cast<unsigned long long>(static_cast<float>(n) * 1048576.f *
                                             fast_exp2(-(j + 0.5f) / s.bins * s.c_hi) + 0.5f);
    };
    unsigned long long all = 0, skip;
    for (int j = tid; j < kBins; j += kThreads) all += guess(j);
    all = block_sum(all, sh.red);
    int b = reach(kBins, max(share_up(p_top, all), 1ull), skip, guess);
    if (b < 0) b = min(b_k, b_min);
    // ---- exact sums: of all candidates, before the bin, in it; then the next bin with entries on the side where the
    // sum is reached, after some turns the middle of those left
    int lo = -1, hi = kBins;                       // it is reached behind lo and before hi
    for (int turn = 0; hi - lo > 1; ++turn) {
      unsigned long long v[3] = {0, 0, 0};
      for_row(row, [&](int i, float x) {
        if (!kept(i, x)) return;
        const unsigned long long w = exact(x);
        const int at = bin_of(s, x);
        v[0] += w;
        v[1] += at < b ? w : 0;
        v[2] += at == b ? w : 0;
      });
      cluster_sums(c, v);
      const unsigned long long target = max(share_up(p_top, v[0]), 1ull);
      if (target > v[1] && target <= v[1] + v[2]) {
        limit = min(limit, settle(c, row, s, top, b, sh.bins[b], target, v[1], kept, exact));
        break;
      }
      const int side = target <= v[1] ? -1 : 1;
      if (side < 0) hi = b; else lo = b;
      b += side;
      while (b > lo && b < hi && sh.bins[b] == 0) b += side;
      if (turn >= 4 || b <= lo || b >= hi) b = (lo + hi) / 2;
    }
  }

  // ---- sums of the kept weights, per warp of consecutive entries
  const int per = ((a.slice + kWarps - 1) / kWarps + 7) & ~7;
  const int w0 = min(row.n, warp * per), w1 = min(row.n, w0 + per);
  unsigned long long own = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const float x = to_float(row.at[i]);
    if (kept(row.first + i, x)) own += exact(x);
  }
  own = warp_sum(own);
  cluster_sync();                                  // (sums[] may still be read for the maximum, or by settle())
  if (lane < static_cast<int>(c.ranks)) remote_store(remote(&sh.sums[c.rank * kWarps + warp], lane), own);
  cluster_sync();
  const int warps = static_cast<int>(c.ranks) * kWarps, me = static_cast<int>(c.rank) * kWarps + warp;
  unsigned long long total = 0, before = 0;
  for (int k = 0; k < warps; ++k) {
    const unsigned long long v = sh.sums[k];
    if (k < me) before += v;
    total += v;
  }
  if (a.tokens) {
    const unsigned long long point = share_down(u, total);         // the token: the first running sum above it
    if (before <= point && point < before + own) {                 // one warp of the cluster
      unsigned long long at = before;
      for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        float x = 0.f;
        unsigned long long w = 0;
        if (i < w1) {
          x = to_float(row.at[i]);
          if (kept(row.first + i, x)) w = exact(x);
        }
        if (__any_sync(0xFFFFFFFFu, w != 0)) {
          const unsigned long long in = warp_scan(w, lane);
          const uint32_t hit = __ballot_sync(0xFFFFFFFFu, w != 0 && at + in > point);
          if (hit) {
            if (lane == __ffs(hit) - 1) a.tokens[r] = row.first + i;
            break;
          }
          at += __shfl_sync(0xFFFFFFFFu, in, 31);
        }
      }
    }
  }
  if (a.probs) {
    float* out = a.probs + static_cast<size_t>(r) * V;
    const float f = static_cast<float>(4398046511104.0 / static_cast<double>(total));       // 2^42 / total
    for (int i = tid; i < row.n; i += kThreads) {
      const float x = to_float(row.at[i]);
      out[row.first + i] = kept(row.first + i, x) ? as_float(weight(s, x, sh.table)) * f : 0.f;
    }
  }
}

template <typename T>
zf_status launch_sample(const SampleArgs& a, bool vec, int ctas, size_t smem, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  const cudaError_t e = vec ? cudaLaunchKernelEx(&cfg, sample_kernel<T, true>, a) : cudaLaunchKernelEx(&cfg, sample_kernel<T, false>, a);
  return e == cudaSuccess ? ZF_OK : ZF_ERR_CUDA;
}

}  // namespace
}  // namespace zf

using namespace zf;

extern "C" zf_status zf_sample_tokens(int32_t rows, int32_t vocab, const void* logits, int32_t logits_type,
                                      int64_t row_stride, const float* uniform, const float* temperature,
                                      const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens,
                                      float* probs, int32_t* status, void* stream) {
  if (rows < 0 || rows > ZF_MAX_SAMPLE_ROWS || vocab < 1 || vocab > ZF_MAX_SAMPLE_VOCAB || row_stride < vocab)
    return ZF_ERR_INVALID_ARGUMENT;
  if (logits_type != ZF_F32 && logits_type != ZF_BF16 && logits_type != ZF_F16) return ZF_ERR_INVALID_ARGUMENT;
  if ((uniform == nullptr) != (tokens == nullptr) || (!tokens && !probs)) return ZF_ERR_INVALID_ARGUMENT;
  if (rows == 0) return ZF_OK;
  const int size = logits_type == ZF_F32 ? 4 : 2;
  if (!logits || (reinterpret_cast<uintptr_t>(logits) & (size - 1))) return ZF_ERR_INVALID_ARGUMENT;
  const void* words[] = {uniform, temperature, top_k, top_p, min_p, tokens, probs, status};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return ZF_ERR_INVALID_ARGUMENT;
  SampleArgs a{};
  a.logits = logits;
  a.uniform = uniform;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.tokens = tokens;
  a.probs = probs;
  a.status = status;
  a.row_stride = row_stride;
  a.rows = rows;
  a.vocab = vocab;
  // CTAs per row: a power of two that brings the grid to 304 CTAs (two per SM) and a slice to 64 KB, with at least
  // 2048 entries each; slices too large for that are kept whole up to 160 KB, and read again from L2 beyond.
  const size_t fixed_smem = (sizeof(Shared) + 15) & ~static_cast<size_t>(15);
  int ctas = 1;
  while (ctas < kMaxCluster && vocab / (2 * ctas) >= 2048 &&
         (static_cast<long long>(rows) * ctas < 304 || static_cast<long long>(vocab) * size / ctas > 65536))
    ctas *= 2;
  a.slice = ((vocab + ctas - 1) / ctas + 7) & ~7;
  const size_t bytes = static_cast<size_t>(a.slice) * size;
  a.cached = bytes <= 163840;
  const size_t smem = fixed_smem + (a.cached ? bytes : 0);
  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZF_ERR_CUDA;
  if (dev < 0 || dev >= 64) return ZF_ERR_UNSUPPORTED;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      const void* kernels[] = {reinterpret_cast<const void*>(sample_kernel<float, true>),
                               reinterpret_cast<const void*>(sample_kernel<float, false>),
                               reinterpret_cast<const void*>(sample_kernel<__nv_bfloat16, true>),
                               reinterpret_cast<const void*>(sample_kernel<__nv_bfloat16, false>),
                               reinterpret_cast<const void*>(sample_kernel<__half, true>),
                               reinterpret_cast<const void*>(sample_kernel<__half, false>)};
      for (const void* k : kernels)
        if (cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(fixed_smem + 163840)) !=
                cudaSuccess)
          return ZF_ERR_CUDA;
      ready[dev] = true;
    }
  }
  a.aligned = aligned16(logits) && (static_cast<size_t>(row_stride) * size) % 16 == 0 && vocab % 8 == 0;
  const bool vec = a.cached || a.aligned;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (logits_type == ZF_F32) return launch_sample<float>(a, vec, ctas, smem, st);
  if (logits_type == ZF_BF16) return launch_sample<__nv_bfloat16>(a, vec, ctas, smem, st);
  return launch_sample<__half>(a, vec, ctas, smem, st);
}
