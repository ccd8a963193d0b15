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
//   2. (top-k, top-p) a histogram of the gap to the maximum, 2048 bins up to 24 temperatures.  It counts: a 32-bit
//      shared-memory atomic per entry, where sums of 64-bit weights would take several, and an exponential each.
//   3. When all that top-k and min-p may keep are at most 512 entries, they are listed in every CTA and ranked by
//      comparing each with each, which settles all filters (a row of 128000 with top-k 22: 20 us instead of 54).
//   4. Otherwise (top-k) the bin with the k-th entry is exact; its entries are listed and ranked.
//   5. (top-p) counts times the bins' middle weights say in which bin the sum is reached; one pass sums the exact
//      weights before it and its neighbours and in each of the three, and lists their entries.  If the guess was wrong
//      by more, the bins beyond are summed.  The entries of the bin are ranked then, and the list also gives what each
//      warp's piece keeps of it.
//   6. (without top-p) sums of the kept weights per warp; then the piece and the entry in which the drawn point lies,
//      and the probabilities.
// A bin with more entries than the list holds is divided again by bits of the places, with exact sums.
//
// What it takes: a row's bytes once from memory are 1.7 to 4 us of the 22 to 40 that a cluster is busy.  The histogram's
// atomics (128000 entries on four CTAs, two CTAs per SM: 7.6 us) and the exponentials of steps 5 and 6 (10 and 7 us for
// 50001 entries), about 55 instructions each, more than half of them on integers, are the rest, with a chain of 8 to 12
// cluster barriers and exchanges of 1 to 2.5 us each.  64 rows of 128000 BF16 logits: 37 us; 320 rows of 50001 FP32
// logits with their probabilities written: 184 us (4.2 rounds of the CTAs that fit).  None of this is the operation's own
// bound: integer weights are needed for the sums and at the border, but every kept entry is given one here, for its
// probability too; equal 16-bit logits are not counted together; and the largest logit alone goes through the histogram.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <climits>
#include <cstddef>
#include <mutex>

#include "zf_device.cuh"
#include "zf_host.h"

namespace zf {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBins = 2048;
constexpr float kRange = 24.f;                     // temperatures that the bins cover
constexpr int kList = 512;                         // entries that are ranked by comparing each with each
constexpr int kSub = 1024;                         // parts in which a crowded interval is divided
static_assert(kList <= kThreads && kSub <= kBins, "an entry per thread; the counts of the parts lie in the bins");
constexpr int kTurns = 20;                         // passes for top-p's bin whose entries are listed on the way

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

// Numbers are rounded to integers and cut to bins by adding 1.5 * 2^23 or 2^23 and reading the low bits: conversion
// instructions run at an eighth of the rate of additions, and four of them per entry were half of a pass's time.
constexpr float kRound = 12582912.f;
constexpr int kRoundBits = 0x4B400000;

struct Weight {
  uint32_t m;                                      // in [2^31 (1 - 2^-11), 2^32)
  int shift;                                       // the weight is m * 2^(shift - 31), shift <= 0
};
__device__ __forceinline__ Weight weight(const Scale& s, float x, const uint32_t* table) {
  // d = x - max exactly as d + e (Knuth's two-sum)
  const float d = __fadd_rn(x, -s.max);
  const float z = __fadd_rn(d, -x);
  const float e = __fadd_rn(__fadd_rn(x, -__fadd_rn(d, -z)), __fadd_rn(-s.max, -z));
  const float y0 = __fmul_rn(d, s.c_hi);
  const float l = __fmaf_rn(d, s.c_hi, -y0) + __fmaf_rn(d, s.c_lo, e * s.c_hi);
  const float y = fmaxf(y0, -4000.f);              // (also a NaN's; the weight is 0 there, whatever l is)
  // y + l = j / 1024 + f, |f| <= 2^-11 and a little
  const float r = __fmaf_rn(y, 1024.f, kRound);
  const float f = __fmaf_rn(__fadd_rn(r, -kRound), -0x1p-10f, y) + l;
  const int j = __float_as_int(r) - kRoundBits;
  // (2^f - 1) 2^31 by its series, to 2^-36 of 2^31
  const float q = f * __fmaf_rn(f, __fmaf_rn(f, 0.0555041087f * 0x1p31f, 0.240226507f * 0x1p31f), 0.693147181f * 0x1p31f);
  const uint32_t t = table[j & 1023];
  const float tf = __int_as_float(static_cast<int>((t >> 8) + 0x3F000000u));      // t 2^-31, cut to 24 bits
  Weight w;
  w.m = t + static_cast<uint32_t>(__float_as_int(__fmaf_rn(q, tf, kRound)) - kRoundBits);
  w.shift = j >> 10;
  return w;
}
// round(2^42 * m * 2^(shift - 31)): m is shifted by 11 + shift
__device__ __forceinline__ unsigned long long fixed(const Weight& w) {
  const int left = 11 + w.shift;
  if (left >= 0) return static_cast<unsigned long long>(w.m) << left;
  const int right = -left - 1;
  return ((right < 32 ? w.m >> right : 0u) + 1) >> 1;
}
// The weight times c (below 2^-20), 0 below 2^-126.
__device__ __forceinline__ float as_float(const Weight& w, float c) {
  return w.shift < -126 ? 0.f : __uint2float_rn(w.m) * c * __int_as_float((127 + w.shift) << 23);
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
  unsigned long long ends[kMaxCluster * kWarps];   // a value of every warp of the cluster (pushed to all CTAs)
  unsigned long long sums[kMaxCluster * kWarps];   // every warp's kept weights
  unsigned long long part[2][kMaxCluster][5];      // per CTA, alternating: sums of a pass
  union {
    alignas(16) Entry list[kList];                 // the same in every CTA
    unsigned long long sub[kSub];                  // weights of the parts of an interval
  };
  uint32_t found_at[3][kList];                     // the CTA's own entries that are to be listed, within its slice
  uint32_t listed[kTurns + 1][3];                  // how many, in every turn
  alignas(16) uint32_t bins[kBins];                            // counts; the cluster's sums in every CTA after fold_bins()
  uint32_t table[1024];
  unsigned long long red[kWarps];
  unsigned long long found[2];                     // a place found by one thread, and the sum before it
};
// (both are read and written 16 bytes at a time)
static_assert(offsetof(Shared, list) % 16 == 0 && offsetof(Shared, bins) % 16 == 0 && sizeof(Shared) % 16 == 0, "layout");

// Whether an entry's weight is min-p's or more, to 32 bits of the weight.  (Few entries are so close: not inlined, as the
// kernel's passes are short and wait for their instructions: 320 x 50001 with probabilities 190 -> 182 us.)
__device__ __noinline__ bool min_keeps(Scale s, float x, float p_min, const uint32_t* table) {
  Weight w = weight(s, x, table);
  if (w.m < 0x80000000u) {
    w.m <<= 1;
    w.shift -= 1;
  }
  int e;
  const float m = frexpf(p_min, &e);               // p_min = m 2^e, m in [0.5, 1)
  const unsigned long long want = static_cast<unsigned long long>(m * 16777216.f) << 8;   // m 2^32
  const int d = w.shift + 1 - e;                   // w = (m_w / 2^32) 2^(shift + 1)
  return d == 0 ? static_cast<unsigned long long>(w.m) >= want : d > 0;
}

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
// The bin is the whole part of this (in the last bin with a NaN).
__device__ __forceinline__ float bin_at(const Scale& s, float x) {
  return fminf((s.max - x) * s.bins, static_cast<float>(kBins - 1));
}
__device__ __forceinline__ int bin_of(const Scale& s, float x) {
  return __float_as_int(__fadd_rz(bin_at(s, x), 8388608.f)) & (kBins - 1);
}

// f(i, step, x) for the entries [w0, w1) of the slice (w0 a multiple of 8), by one warp: four per lane at a time, i and
// every step-th from there, so that their arithmetic overlaps; NaN behind the end.  All lanes call f together.
template <typename T, bool kVec, typename F>
__device__ __forceinline__ void for_fours(const Row<T, kVec>& r, int w0, int w1, F&& f) {
  const int lane = threadIdx.x & 31;
  for (int i0 = w0; i0 < w1; i0 += 128) {
    float x[4];
    if (kVec) {
      struct alignas(4 * sizeof(T)) Pack {
        T v[4];
      };
      const int i = i0 + 4 * lane;
      Pack p{};
      if (i < w1) p = *reinterpret_cast<const Pack*>(r.at + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = i + e < w1 ? to_float(p.v[e]) : CUDART_NAN_F;
      f(i, 1, x);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = i0 + lane + 32 * e < w1 ? to_float(r.at[i0 + lane + 32 * e]) : CUDART_NAN_F;
      f(i0 + lane, 32, x);
    }
  }
}

struct Ctx {
  Shared* sh;
  uint32_t rank, ranks;
  int flip;                                        // which part[] the next exchange uses
  int index_bits;                                  // of the vocabulary
};

// The largest of all threads' values.
__device__ __forceinline__ unsigned long long block_max(unsigned long long* red, unsigned long long v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) v = max(v, red[w]);
  return v;
}

// Sums of five values over the warp (in mine), and over the cluster (in v; every thread gets them).
__device__ __forceinline__ void cluster_sums(Ctx& c, unsigned long long (&v)[5], unsigned long long (&mine)[5]) {
  Shared& sh = *c.sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ unsigned long long red[5][kWarps];
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    mine[k] = warp_sum(v[k]);
    if (lane == 0) red[k][warp] = mine[k];
  }
  __syncthreads();
  if (warp < 5) {
    const unsigned long long s = warp_sum(lane < kWarps ? red[warp][lane] : 0);
    if (lane < static_cast<int>(c.ranks)) remote_store(remote(&sh.part[c.flip][c.rank][warp], lane), s);
  }
  cluster_sync();
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    v[k] = 0;
    for (uint32_t r = 0; r < c.ranks; ++r) v[k] += sh.part[c.flip][r][k];
  }
  c.flip ^= 1;
}

// The cluster's sums of bins[0 .. n) into every CTA's bins (n a multiple of 4).
__device__ __forceinline__ void fold_bins(Ctx& c, uint32_t* bins, int n) {
  if (c.ranks == 1) {
    __syncthreads();
    return;
  }
  cluster_sync();
  const int quads = n / 4, per = (quads + static_cast<int>(c.ranks) - 1) / static_cast<int>(c.ranks);
  const int lo = static_cast<int>(c.rank) * per, hi = min(quads, lo + per);
  for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
    uint32_t s[4] = {0, 0, 0, 0};
    for (uint32_t r0 = 0; r0 < c.ranks; r0 += 2) {   // (ranks are a power of two; two loads under way)
      uint32_t x[2][4];
#pragma unroll
      for (uint32_t d = 0; d < 2; ++d)
        asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[d][0]), "=r"(x[d][1]), "=r"(x[d][2]), "=r"(x[d][3])
                     : "r"(remote(&bins[4 * i], r0 + d))
                     : "memory");
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += x[0][e] + x[1][e];
    }
    for (uint32_t r = 0; r < c.ranks; ++r)
      asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(remote(&bins[4 * i], r)), "r"(s[0]), "r"(s[1]),
                   "r"(s[2]), "r"(s[3])
                   : "memory");
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

// The entries that the CTAs have found (found_at, listed) become every CTA's list: their number.  entry(j) is the entry
// at place j of the slice.  Called behind a cluster barrier, ends with one.
template <typename MakeEntry>
__device__ __forceinline__ int share_list(Ctx& c, int turn, int which, MakeEntry&& entry) {
  Shared& sh = *c.sh;
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t n = lane < c.ranks ? remote_load32(remote(&sh.listed[turn][which], lane)) : 0;
  const uint32_t all = __reduce_add_sync(0xFFFFFFFFu, n), first = __reduce_add_sync(0xFFFFFFFFu, lane < c.rank ? n : 0);
  const uint32_t own = sh.listed[turn][which];
  for (uint32_t k = threadIdx.x; k < own && first + k < kList; k += kThreads) {
    const Entry e = entry(static_cast<int>(sh.found_at[which][k]));
    for (uint32_t r = 0; r < c.ranks; ++r)
      asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(remote(&sh.list[first + k], r)), "l"(e.at), "l"(e.w)
                   : "memory");
  }
  cluster_sync();
  return static_cast<int>(min(all, static_cast<uint32_t>(kList)));
}
// Among the n listed entries: the place at which the running sum along the order reaches target (>= 1), and that sum
// without it (the last place when it is not reached).  Every CTA finds it for itself.
__device__ __forceinline__ unsigned long long rank_list(Ctx& c, int n, unsigned long long target, unsigned long long& before) {
  Shared& sh = *c.sh;
  if (threadIdx.x == 0) {
    sh.found[0] = ~0ull;
    sh.found[1] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Entry own = sh.list[i];
    unsigned long long sum = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const Entry o = sh.list[j];
      if (o.at <= own.at) sum += o.w;
    }
    if (sum >= target && sum - own.w < target) {
      sh.found[0] = own.at;
      sh.found[1] = sum - own.w;
    }
  }
  __syncthreads();
  before = sh.found[1];
  const unsigned long long at = sh.found[0];
  __syncthreads();                                 // (the words are used again, by the guess of top-p's bin too)
  return at;
}
// One more entry that is to be listed.
__device__ __forceinline__ void append(Ctx& c, int turn, int which, int at) {
  const uint32_t k = atomicAdd(&c.sh->listed[turn][which], 1u);
  if (k < kList) c.sh->found_at[which][k] = static_cast<uint32_t>(at);
}

// The place at which the running sum of value(x) (1 or a weight; entries that are not in are skipped) along the order
// reaches target, where it is known to lie in bin b, before which the sum is `before` (updated to the sum before the
// place).  n: an upper bound of the entries in the bin.  listed: how many they are if they are all in the list then, or
// -1; complete: whether the CTAs have found them already.
template <typename T, bool kVec, typename In, typename Val>
__device__ __forceinline__ unsigned long long settle(Ctx& c, const Row<T, kVec>& row, const Scale& s, uint32_t top, int b,
                                                     uint32_t n, int turn, int which, unsigned long long target, unsigned long long& before,
                                                     int& listed, bool complete, In&& in, Val&& value) {
  Shared& sh = *c.sh;
  // an interval of places, the index moved up to the gap: dividing it by bits then comes to the index sooner
  unsigned long long lo = 0, hi = ~0ull;
  auto close = [&](int i, float x) { return static_cast<unsigned long long>(top - order_of(x)) << c.index_bits | static_cast<uint32_t>(i); };
  const float g0 = static_cast<float>(b), g1 = static_cast<float>(b + 1);
  auto in_bin = [&](float x) {
    const float g = bin_at(s, x);
    return g >= g0 && g < g1;
  };
  const bool whole = n <= kList;
  listed = -1;
  if (n > kList) {
    // the interval's ends, then parts of it by their bits
    unsigned long long mn = ~0ull, mx = 0;
    for_row(row, [&](int i, float x) {
      if (in_bin(x) && in(i, x)) {
        const unsigned long long p = close(i, x);
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
      if ((threadIdx.x & 31) < c.ranks) remote_store(remote(&sh.ends[me], threadIdx.x & 31), pass ? mx : mn);
      cluster_sync();
      for (uint32_t k = 0; k < c.ranks * kWarps; ++k) {
        const unsigned long long v = sh.ends[k];
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
        if (!in_bin(x) || !in(i, x)) return;
        const unsigned long long p = close(i, x);
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
    if (lo >= hi) return (lo >> c.index_bits) << 32 | (lo & ((1ull << c.index_bits) - 1));
    cluster_sync();                                // (the list lies over the parts)
  }
  if (!complete) {
    for_row(row, [&](int i, float x) {
      if (!in_bin(x) || !in(i, x)) return;
      const unsigned long long p = close(i, x);
      if (p >= lo && p <= hi) append(c, turn, which, i - row.first);
    });
    cluster_sync();
  }
  const int many = share_list(c, turn, which, [&](int j) {
    const float x = to_float(row.at[j]);
    return Entry{place(top, x, row.first + j), value(x)};
  });
  if (whole) listed = many;
  unsigned long long inner;
  const unsigned long long at = rank_list(c, many, target - before, inner);
  before += inner;
  return at;
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  T* cache = reinterpret_cast<T*>(raw + ((sizeof(Shared) + 15) & ~static_cast<size_t>(15)));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Ctx c{&sh, cluster_rank(), cluster_size(), 0, 32 - __clz(a.vocab)};
  const int r = blockIdx.x / c.ranks, V = a.vocab;
  for (int k = tid; k < 1024; k += kThreads) sh.table[k] = kExp2.v[k];
  if (tid < (kTurns + 1) * 3) sh.listed[tid / 3][tid % 3] = 0;
  allow_next_grid();
  wait_prior_grid();
  cluster_sync();                                  // all CTAs run before their shared memory is written

  // ---- the row, and its maximum
  Row<T, kVec> row;
  row.first = min(V, static_cast<int>(c.rank) * a.slice);
  row.n = min(V - row.first, a.slice);
  row.at = static_cast<const T*>(a.logits) + static_cast<long long>(r) * a.row_stride + row.first;
  float most = -CUDART_INF_F;                      // (fmaxf passes NaN by)
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
          if (i < row.n) {
            *reinterpret_cast<uint4*>(cache + i) = v[k];
#pragma unroll
            for (int e = 0; e < kPer; ++e) most = fmaxf(most, to_float(reinterpret_cast<const T*>(&v[k])[e]));
          }
        }
      }
    } else {
#pragma unroll 8
      for (int i = tid; i < row.n; i += kThreads) {
        const T x = row.at[i];
        cache[i] = x;
        most = fmaxf(most, to_float(x));
      }
    }
    row.at = cache;
    __syncthreads();
  } else {
    for_row(row, [&](int, float x) { most = fmaxf(most, x); });
  }
  const uint32_t order = __reduce_max_sync(0xFFFFFFFFu, order_of(most));
  if (lane < static_cast<int>(c.ranks)) remote_store(remote(&sh.ends[c.rank * kWarps + warp], lane), order);
  cluster_sync();
  uint32_t top = 0;
  for (int k = lane; k < static_cast<int>(c.ranks) * kWarps; k += 32) top = max(top, static_cast<uint32_t>(sh.ends[k]));
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
  // A logit above sure is kept and one below out is not; between them its place, and min-p by its weight, decide.
  float sure = -CUDART_INF_F, out = -CUDART_INF_F;
  if (by_min) {
    const float gap = -log2f(p_min) / s.c_hi;
    sure = __fsub_ru(s.max, gap * 0.99999f);
    out = __fsub_rd(s.max, gap * 1.00001f);
  }
  auto above_min = [&](float x) { return min_keeps(s, x, p_min, sh.table); };
  auto bound = [&](unsigned long long last) {      // nothing behind this place is kept
    if (last >= limit) return;
    limit = last;
    const uint32_t o = top - static_cast<uint32_t>(last >> 32);
    const float x = __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
    sure = fmaxf(sure, x);
    out = fmaxf(out, x);
  };
  // the last bin with entries that top-k and min-p may keep, and whether all up to it can be listed
  const float g_min = by_min ? fminf(-log2f(p_min) / s.c_hi * s.bins, static_cast<float>(kBins - 1)) : kBins - 1;
  const int b_min = static_cast<int>(g_min), b_end = min(b_k, by_min ? b_min + 1 : kBins - 1);
  int few_entries = 0;
  if ((by_k || by_p) && b_end < kBins - 1) {
    constexpr int kOwn = kBins / kThreads;
    uint32_t n = 0;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) n += tid * kOwn + k <= b_end ? sh.bins[tid * kOwn + k] : 0;
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0) sh.red[warp] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < kWarps; ++w) n += static_cast<uint32_t>(sh.red[w]);
    few_entries = n <= kList ? static_cast<int>(n) : 0;
    __syncthreads();
  }
  if (by_k && few_entries == 0) {
    // settle() overwrites the bins when it divides: what top-p needs of them is kept only if it does not
    int listed;
    unsigned long long before = before_k;
    bound(settle(c, row, s, top, b_k, n_k, kTurns, 0, static_cast<unsigned long long>(k_top), before, listed, false,
                 [&](int, float) { return true; }, [](float) { return 1ull; }));
  }
  auto kept = [&](int i, float x) {                // (a NaN is not, its weight is 0)
    return x > sure || (x >= out && place(top, x, i) <= limit && (!by_min || above_min(x)));
  };
  // this warp's consecutive entries of the slice, and its sum of kept weights
  const int per = ((a.slice + kWarps - 1) / kWarps + 7) & ~7;
  const int w0 = min(row.n, warp * per), w1 = min(row.n, w0 + per);
  unsigned long long own = 0;
  bool known = false;
  if (few_entries > 0) {
    // ---- all that may be kept is listed: its places and running sums along the order say what is
    const float g_end = static_cast<float>(b_end + 1);
    for_row(row, [&](int i, float x) {
      if (bin_at(s, x) < g_end) append(c, kTurns, 0, i - row.first);
    });
    cluster_sync();
    const int n = share_list(c, kTurns, 0, [&](int j) {
      const float x = to_float(row.at[j]);
      return Entry{place(top, x, row.first + j), exact(x)};
    });
    // (one entry per thread)
    Entry e{~0ull, 0};
    unsigned long long sum = 0;
    bool in = false;
    if (tid < n) {
      e = sh.list[tid];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const Entry o = sh.list[j];
        if (o.at <= e.at) {
          sum += o.w;
          ++rank;
        }
      }
      const uint32_t o = top - static_cast<uint32_t>(e.at >> 32);
      const float x = __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
      in = (!by_k || rank <= k_top) && (x > sure || (x >= out && (!by_min || above_min(x))));
    }
    const unsigned long long all = block_max(sh.red, in ? sum : 0);
    const unsigned long long target = by_p ? max(share_up(p_top, all), 1ull) : all;
    bound(block_max(sh.red, in && sum - e.w < target ? e.at : 0));
    const uint32_t first = row.first + w0, many = w1 - w0;
    for (int k = lane; k < n; k += 32) {
      const Entry o = sh.list[k];
      if (o.at <= limit && static_cast<uint32_t>(o.at) - first < many) own += o.w;
    }
    own = warp_sum(own);
    known = true;
  } else if (by_p) {
    if (by_k && n_k > kList) {                     // the counts again
      for (int k = tid; k < kBins; k += kThreads) sh.bins[k] = 0;
      __syncthreads();
      for_row(row, [&](int, float x) { atomicAdd(&sh.bins[bin_of(s, x)], 1u); });
      __syncthreads();
      fold_bins(c, sh.bins, kBins);
    }
    // middle weights of the bins, of those that top-k or min-p cuts the part that is kept, none of the last; kBins /
    // kThreads per thread
    constexpr int kOwn = kBins / kThreads;
    float part[kOwn], mine = 0.f;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const int j = tid * kOwn + k;
      const float n = j > b_k || j > b_min || j == kBins - 1 ? 0.f
                      : j == b_k && by_k                     ? static_cast<float>(k_top - before_k)
                      : j == b_min && by_min                 ? static_cast<float>(sh.bins[j]) * (g_min - static_cast<float>(j))
                                                             : static_cast<float>(sh.bins[j]);
      mine += n * fast_exp2(-(j + 0.5f) / s.bins * s.c_hi);
      part[k] = mine;
    }
    float in = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float x = __shfl_up_sync(0xFFFFFFFFu, in, d);
      if (lane >= d) in += x;
    }
    float* ends = reinterpret_cast<float*>(sh.red);
    int* guess = reinterpret_cast<int*>(sh.found);
    if (lane == 31) ends[warp] = in;
    if (tid == 0) *guess = min(b_k, b_min);
    __syncthreads();
    float lead_in = in - mine, all = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      lead_in += w < warp ? ends[w] : 0.f;
      all += ends[w];
    }
#pragma unroll
    for (int k = kOwn - 1; k >= 0; --k) {            // the first bin whose running sum reaches the point
      const float before_bin = lead_in + (k > 0 ? part[k - 1] : 0.f);
      if (before_bin < p_top * all && lead_in + part[k] >= p_top * all) atomicMin(guess, tid * kOwn + k);
    }
    __syncthreads();
    int b = *guess;
    __syncthreads();
    // ---- exact sums: of all candidates, before the bins b - 1 .. b + 1, in each of these, whose entries are listed on the
    // way (lists of their own for every turn).  When the sum is reached in none of them, the next bins with entries
    // on the side where it is, after some turns the middle of those left; only what lies between is summed then.
    int lo = -1, hi = kBins;                       // it is reached behind lo and before hi
    unsigned long long all_sum = 0, base = 0, base_lead = 0;       // of all; up to lo; of this warp's up to lo
    for (int turn = 0; hi - lo > 1; ++turn) {
      bool few[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) few[k] = turn < kTurns && sh.bins[min(max(b - 1 + k, 0), kBins - 1)] <= kList;
      unsigned long long v[5] = {0, 0, 0, 0, 0};
      const float g0 = static_cast<float>(lo + 1), g1 = static_cast<float>(b - 1), g2 = static_cast<float>(b),
                  g3 = static_cast<float>(b + 1), g4 = static_cast<float>(b + 2);
      for_fours(row, w0, w1, [&](int i, int step, const float (&x)[4]) {
        bool in[4], any = false;
        float g[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[e] = bin_at(s, x[e]);
          in[e] = kept(row.first + i + step * e, x[e]) && (turn == 0 || (g[e] >= g0 && g[e] < g4));
          any |= in[e];
        }
        if (!__any_sync(0xFFFFFFFFu, any)) return;
        bool window = false;
        unsigned long long w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = exact(x[e]);
          v[0] += in[e] ? w[e] : 0;
          v[1] += in[e] && g[e] < g1 ? w[e] : 0;
          window |= in[e] && g[e] >= g1 && g[e] < g4;
        }
        if (!window) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!(in[e] && g[e] >= g1 && g[e] < g4)) continue;
          const int k = g[e] < g2 ? 0 : g[e] < g3 ? 1 : 2;
          v[2] += k == 0 ? w[e] : 0;
          v[3] += k == 1 ? w[e] : 0;
          v[4] += k == 2 ? w[e] : 0;
          if (k == 0 ? few[0] : k == 1 ? few[1] : few[2])
            append(c, turn, k, i + step * e);
        }
      });
      unsigned long long mine[5];
      cluster_sums(c, v, mine);
      unsigned long long lead = base_lead + mine[1];           // this warp's weights before the bins
      if (turn == 0) all_sum = v[0];
      const unsigned long long target = max(share_up(p_top, all_sum), 1ull);
      unsigned long long before = base + v[1];
      if (target > before && target <= before + v[2] + v[3] + v[4]) {
        int in = 0;
        if (target > before + v[2]) {
          before += v[2];
          lead += mine[2];
          in = 1;
          if (target > before + v[3]) {
            before += v[3];
            lead += mine[3];
            in = 2;
          }
        }
        int listed;
        const bool ready = in == 0 ? few[0] : in == 1 ? few[1] : few[2];
        const unsigned long long last = settle(c, row, s, top, b - 1 + in, sh.bins[b - 1 + in], ready ? turn : kTurns,
                                               ready ? in : 1, target, before, listed, ready, kept, exact);
        bound(last);
        known = ready && listed >= 0;
        if (known) {
          // the bin's entries are all listed: no pass for the sums
          const uint32_t first = row.first + w0, many = w1 - w0;
          own = 0;
          for (int k = lane; k < listed; k += 32) {
            const Entry e = sh.list[k];
            if (e.at <= limit && static_cast<uint32_t>(e.at) - first < many) own += e.w;
          }
          own = warp_sum(own) + lead;
        }
        break;
      }
      int side = -1;
      if (target <= before) {
        hi = b - 1;
      } else {
        side = 1;
        lo = b + 1;
        base = before + v[2] + v[3] + v[4];
        base_lead = lead + mine[2] + mine[3] + mine[4];
      }
      b += 2 * side;
      while (b > lo && b < hi && sh.bins[b] == 0) b += side;
      b += side;
      if (turn >= 4 || b <= lo || b >= hi) b = (lo + hi) / 2;
    }
  }

  // ---- sums of the kept weights, per warp
  if (!known) {
    own = 0;
    for_fours(row, w0, w1, [&](int i, int step, const float (&x)[4]) {
      bool in[4], any = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) any |= in[e] = kept(row.first + i + step * e, x[e]);
      if (!__any_sync(0xFFFFFFFFu, any)) return;
#pragma unroll
      for (int e = 0; e < 4; ++e) own += in[e] ? exact(x[e]) : 0;
    });
    own = warp_sum(own);
  }
  if (lane < static_cast<int>(c.ranks)) remote_store(remote(&sh.sums[c.rank * kWarps + warp], lane), own);
  cluster_sync();
  const int warps = static_cast<int>(c.ranks) * kWarps, me = static_cast<int>(c.rank) * kWarps + warp;
  unsigned long long total = 0, before = 0;
  for (int k = lane; k < warps; k += 32) {
    const unsigned long long v = sh.sums[k];
    total += v;
    before += k < me ? v : 0;
  }
  total = warp_sum(total);
  before = warp_sum(before);
  if (a.tokens) {
    const unsigned long long point = share_down(u, total);         // the token: the first running sum above it
    if (before <= point && point < before + own) {                 // one warp of the cluster
      unsigned long long at = before;
      for (int i0 = w0; i0 < w1; i0 += 128) {
        unsigned long long w[4], four = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + 4 * lane + e;
          const float x = i < w1 ? to_float(row.at[i]) : CUDART_NAN_F;
          w[e] = kept(row.first + i, x) ? exact(x) : 0;
          four += w[e];
        }
        if (!__any_sync(0xFFFFFFFFu, four != 0)) continue;
        const unsigned long long in = warp_scan(four, lane);
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, at + in > point);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            at += in - four;
            int e = 0;
            while (e < 3 && at + w[0] <= point) {    // (one of the four passes the point)
              at += w[0];
              w[0] = e == 0 ? w[1] : e == 1 ? w[2] : w[3];
              ++e;
            }
            a.tokens[r] = row.first + i0 + 4 * lane + e;
          }
          break;
        }
        at += __shfl_sync(0xFFFFFFFFu, in, 31);
      }
    }
  }
  if (a.probs) {
    float* to = a.probs + static_cast<size_t>(r) * V;
    const float f = static_cast<float>(2048.0 / static_cast<double>(total));       // 2^(42 - 31) / total
    for (int i0 = tid - lane; i0 < row.n; i0 += 4 * kThreads) {
      float x[4];
      bool in[4], any = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + lane + kThreads * e;
        x[e] = i < row.n ? to_float(row.at[i]) : CUDART_NAN_F;
        any |= in[e] = kept(row.first + i, x[e]);
      }
      any = __any_sync(0xFFFFFFFFu, any);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + lane + kThreads * e;
        const float p = any ? as_float(weight(s, x[e], sh.table), f) : 0.f;
        if (i < row.n) to[row.first + i] = in[e] ? p : 0.f;
      }
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
  // CTAs per row: a power of two, as long as all rows' CTAs run at once (two per SM; clusters of 16 find room for about
  // one per SM) and each has 2560 entries; and so many that a slice is no more than 72 KB (two CTAs' fit an SM then),
  // where eight are enough for slices of 160 KB, which are still kept whole (beyond, they are read again from L2).
  // Measured with top-p, us for 1, 2, 4, 8, 16 CTAs: 32000 BF16, 8 rows 42, 29, 22, 19, 23, 64 rows 45, 37, 29, 44, 100,
  // 256 rows 60, 72, 96, 155, 360; 8192, 32 rows 18, 17, 18, 20, 55; 128000, 1 row -, 80, 47, 31, 28, 64 rows -, 84, 75, 92,
  // 151; 256000 FP32, 128 rows 423 with 8 (slices of 128 KB), 486 with 16.
  const size_t fixed_smem = (sizeof(Shared) + 15) & ~static_cast<size_t>(15);
  int ctas = 1;
  while (ctas < kMaxCluster) {
    const long long all = static_cast<long long>(rows) * 2 * ctas, bytes = static_cast<long long>(vocab) * size / ctas;
    if (!(vocab / (2 * ctas) >= 2560 && all <= (2 * ctas == kMaxCluster ? 152 : 304)) && bytes <= (ctas < 8 ? 73728 : 163840)) break;
    ctas *= 2;
  }
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
