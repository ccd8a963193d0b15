// zf_q4_decode_attn: split-KV decode attention over the 4-bit paged cache (one or several new tokens
// per request), and its split-result merge.
//
// Mathematics.  K and V are code * s (16-channel blocks, e2m1 codes of two significant bits, e4m3
// scales of four): every product code * s has at most six significant bits and is exact in fp16, so
// the operands of the matrix instructions are the stored values themselves.  q (BF16) is brought into
// fp16 by a power of two per row, which its scores take back: values down to 2^-28 of the row's largest exponent
// are exact, smaller ones fall on a grid of 2^-35 (off by 2^-36 at most).  Scores, running maximum and sum
// and the output are float32.  The softmax weights p (times 2^7, so that the remainder of a small weight
// stays clear of fp16's subnormals) are split into an fp16 high part and an fp16 remainder, two MMAs: off by
// at most 2^-22 of the weight or, where parts are subnormal, 2^-30 of the range's largest (which is above 2^6).
//
// Work split.  The 16-token records of all (request, kv head, column slice) pairs, laid end to end, are
// cut into one equal contiguous range per warp of the grid (one CTA per SM).  A warp goes through its
// range on its own: it walks the pairs, works out 32 records' addresses at a time, stages its pair's query rows,
// streams units of two records into two private shared-memory stages (one 2304-byte bulk copy per
// record, the next unit's under way while it works on this one) and, where a pair ends or its range
// does, writes the result (a pair that lies within the range) or a partial: its weighted sum of
// values, maximum and sum.  There is no barrier after the prologue and no combine between warps; a
// range has at most two partials (its first and its last pair).  A second kernel merges them.
// (With a CTA per item, a metadata warp and a combine of the warps' states at each item's end, the
// barriers and the part-filled last rounds cost 4 us per item: 91.3 us at the ragged 64-request workload.)
//
// Fragments.
//  * K: a lane's A fragments of all eight k-steps are 16 contiguous bytes of a token's row (the order
//    of channels within the k-steps is free as long as q follows it), two 16-byte reads per record, and
//    it meets two scale blocks per token, four scale bytes in one 4-byte read.
//  * V: a lane's rows are the 16 channels of one block (eight m-tiles x two rows), so it needs one scale
//    per token: four tokens' codes in four 8-byte reads, their scales in one 4-byte read.  The codes
//    of two tokens are interleaved by nibble, so that one conversion gives a register of the
//    operand (two tokens, one channel).
//  * e2m1 pairs become half pairs in one conversion, and one multiplication applies the scale.
//
// Bound.  Up to 8 columns no unit is near its limit (issue slots 62 to 65% busy, ALU 52 to 57%, DRAM 54 to 62%):
// 340 and 369 instructions per record, many of half rate, beside the copies; 106 and 127 cycles per record and
// SM, the copies alone 101.  Wider: the matrix instructions, each of which holds its scheduler for 9.4 cycles and
// overlaps other work only in part (28 columns: 96 per record, 226 of 430 cycles).  The 5th-generation tensor
// cores do not pay here: with K in tensor memory, V^T in shared memory and a product per 128 tokens the softmax's
// chain of dependent steps sets the pace, 2700 to 3100 cycles per 128 tokens for 16 to 32 columns alike (28
// columns, 32 requests of 8192 tokens 87 us against 95 here, of 2048 tokens and 64 requests 125 against 105, of
// 128 tokens 41 against 27).
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <climits>
#include <mutex>

#include "zf_attn_common.cuh"
#include "zf_q4.cuh"

namespace zf {

namespace {

constexpr int kUnitTiles = 2;                            // records per stage
constexpr int kStageQ4 = kUnitTiles * kQ4Record;         // 4608
constexpr int kQ4QRowBytes = 320;                        // q row in shared memory (see store_q_row)
constexpr int kFewPartials = 20;                         // see range_length
constexpr float kUnseen = -3e38f;                        // a maximum before any visible score: finite, below them all
constexpr float kPShift = 7.f;                           // weights are 2^7 times their usual size

// Warps per CTA by the number of 8-column tiles of a pass (kNT), from the registers they need (128, 168
// and, for three and four tiles, 255 per thread).  Only the instances for up to 4 columns need no more than that;
// the others spill (bytes stored: 5 to 8 columns 4 to 8, two tiles 24, three 28, four 104).
template <int kNT>
struct Q4Cfg {
  static constexpr int kWarps = kNT == 1 ? 16 : kNT == 2 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kCols = 8 * kNT;
};

struct Q4AttnArgs {
  const uint8_t* records;
  int32_t* status;
  const uint16_t* q;
  const int32_t* page_table;
  const int32_t* seq_lens;
  float* out;
  float* lse;
  float* part_o;              // [range][2][columns][128]: partials of a range's first and last pair
  float2* part_ml;            // [range][2][columns]: their maximum (log2 units) and sum
  int32_t* prefix;            // [batch + 1] records of the requests before each; [batch + 1] has the range length
  int32_t batch, hq, hkv, group, slices, page_size, num_pages, max_pages;
  int32_t tokens;             // new tokens per request T: query head qh = head * T + token (hq, group count them)
  float scale_log2;           // softmax scale * log2(e) * scales of the decoding
  float v_factor;
  uint64_t wait_limit_ns;     // limit of the waits for copies (kWaitTimeoutNs; tests shorten it)
  int32_t hold_copies;        // tests: every warp's first wait runs out (see the barriers' initial counts)
};

// What a warp keeps of the query columns of its current pair.
template <int kNT>
struct Q4Columns {
  float scale[8 * kNT];          // score factor
  int at[8 * kNT];               // row within the request's query rows
  int token[8 * kNT];            // new token
};

struct Q4Smem {
  size_t stages, qbuf, cols, bars, prefix, total;
};

template <int kNT>
__host__ __device__ inline Q4Smem q4_smem(int batch) {
  using C = Q4Cfg<kNT>;
  Q4Smem s;
  size_t at = 0;
  s.stages = at; at += static_cast<size_t>(C::kWarps) * kWarpStages * kStageQ4;
  s.qbuf = at; at += static_cast<size_t>(C::kWarps) * C::kCols * kQ4QRowBytes;
  s.cols = at; at += C::kWarps * sizeof(Q4Columns<kNT>);
  s.bars = at; at += static_cast<size_t>(C::kWarps) * kWarpStages * 8;
  s.prefix = at; at += static_cast<size_t>(batch + 1) * 4;
  s.total = (at + 127) & ~static_cast<size_t>(127);
  return s;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same into a fresh accumulator.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 8x8 transpose of 16-bit values (as transpose8x8, free to move between other instructions).
__device__ __forceinline__ uint32_t flip8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two floats in a register pair, and the packed additions and fused multiply-adds on them.
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// d += s, rounded to nearest.  The matrix instructions cut their float sums off instead, a bias that
// grows along a chain of accumulations, so a chain is one unit long and is added to the output here: a quarter of
// the error against 64 bits at the long-context workload (now 5.3e-7 of the outputs' root mean square; a plain
// float32 form 4.7e-7), for 2 to 8% of the time.
__device__ __forceinline__ void add4(float (&d)[4], const float (&s)[4]) {
  const F2 a = add2(F2{d[0], d[1]}, F2{s[0], s[1]}), b = add2(F2{d[2], d[3]}, F2{s[2], s[3]});
  d[0] = a.x;
  d[1] = a.y;
  d[2] = b.x;
  d[3] = b.y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The query rows of a pair (query heads h0 .. h0 + nh - 1 of request b), by one warp, into shared memory as fp16:
// each row times a power of two that brings its largest exponent to 11; its factor takes that back.  Rows
// past nh are zero.  All loads come before the first store, so they are under way together.  (Ordinary loads, at
// the same times as read-only ones, which need q to stay as it is for the whole grid: this grid starts while the
// kernel ahead of it may still be writing q.)  Channel c = 32 t + 8 j + e goes to byte 64 j + 16 t + 2 e: lane
// t's words of k-steps 2j, 2j+1 are 16 bytes, and the rows' stride spreads a warp's reads over the banks.  A
// warp takes four rows one by one (one maximum over the lanes each), more two by two.  (Rows one by one, and a
// division per column here, for the mask and for the result: 64 requests of 512 tokens, 32 columns 61.2 us
// instead of 51.4; four rows two by two: the long-context workload 110.8 instead of 109.7.)
template <int kNT, bool kFold>
__device__ __forceinline__ void stage_q(const Q4AttnArgs& a, int b, int h0, int nh, uint8_t* qb, Q4Columns<kNT>& cols,
                                        int lane) {
  static_assert(!kFold || kNT == 1, "four columns");
  constexpr int kRows = kFold ? 4 : 8 * kNT;
  int rel = 0;
  if (lane < 8 * kNT) {
    const int qh = h0 + min(kFold ? lane & 3 : lane, nh - 1);
    const int h = a.tokens == 1 ? qh : qh / a.tokens, tok = qh - h * a.tokens;
    rel = tok * (a.tokens == 1 ? a.hq : a.hq / a.tokens) + h;
    cols.at[lane] = rel;
    cols.token[lane] = tok;
  }
  const bool negate = a.scale_log2 < 0.f;
  // a row's factor from the largest magnitude among its values (their bits)
  auto factor = [&](uint32_t big, float& s) {
    const int k = min(138 - static_cast<int>(big >> 7), 126);           // (big >> 7: biased exponent)
    // positive, so that the largest raw score has the largest score, and -inf stays one
    s = fmaxf(__int_as_float((127 - k) << 23) * fabsf(a.scale_log2), 1e-37f);
    return __int_as_float(((127 + k) << 23) | (negate ? 0x80000000 : 0));
  };
  if constexpr (kFold) {
    const uint32_t* base = reinterpret_cast<const uint32_t*>(a.q + static_cast<size_t>(b) * a.hq * ZF_HEAD_DIM) + lane;
    uint32_t v[kRows][2];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const uint32_t* src = base + static_cast<size_t>(__shfl_sync(0xFFFFFFFFu, rel, r)) * (ZF_HEAD_DIM / 2);
      v[r][0] = r < nh ? src[0] : 0u;
      v[r][1] = r < nh ? src[32] : 0u;
    }
    uint8_t* dst = qb + 64 * ((lane >> 2) & 3) + 16 * (lane >> 4) + 4 * (lane & 3);        // channel 2 lane; 2 lane + 64 is 32 on
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const uint32_t m2 = __vmaxu2(v[r][0] & 0x7FFF7FFFu, v[r][1] & 0x7FFF7FFFu);
      float s;
      const float f = factor(__reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16)), s);
#pragma unroll
      for (int c = 0; c < 2; ++c) {                          // (columns 4 to 7 repeat 0 to 3)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<uint32_t*>(dst + (r + 4 * c) * kQ4QRowBytes + 32 * h) =
              pack_f16x2(bf16lo_to_f32(v[r][h]) * f, bf16hi_to_f32(v[r][h]) * f);
        if (lane == 0) cols.scale[r + 4 * c] = s;
      }
    }
  } else {
    const int m = lane & 15;                                   // channels 8m .. 8m + 7
    const uint4* base = reinterpret_cast<const uint4*>(a.q + static_cast<size_t>(b) * a.hq * ZF_HEAD_DIM) + m;
    uint8_t* dst = qb + 64 * (m & 3) + 16 * (m >> 2);
    uint4 v[kRows / 2];
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) {
      const int r = 2 * i + (lane >> 4);
      const size_t row = static_cast<size_t>(__shfl_sync(0xFFFFFFFFu, rel, r)) * (ZF_HEAD_DIM / 8);
      v[i] = r < nh ? base[row] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) {
      const int r = 2 * i + (lane >> 4);
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t big = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) big = __vmaxu2(big, __shfl_xor_sync(0xFFFFFFFFu, big, d));
      float s;
      const float f = factor(max(big & 0xFFFFu, big >> 16), s);
      uint32_t y[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) y[x] = pack_f16x2(bf16lo_to_f32(w[x]) * f, bf16hi_to_f32(w[x]) * f);
      *reinterpret_cast<uint4*>(dst + r * kQ4QRowBytes) = make_uint4(y[0], y[1], y[2], y[3]);
      if (m == 0) cols.scale[r] = s;
    }
  }
}

// Records per range: an equal share of the total, but enough that a pair's partials stay few (the square of
// the length times kFewPartials at least the mean records of a pair; one request of 8192 tokens, 8 kv
// heads: 26.0 us with the equal share of 2 records and up to 256 partials, 10.7 with 6 and 86); an even
// number, so that units are whole.
__host__ __device__ inline int range_length(long long total, int ranges, int mean) {
  int W = static_cast<int>((total + 2LL * ranges - 1) / (2LL * ranges)) * 2;
  while (W > 0 && static_cast<long long>(W) * W * kFewPartials < mean) W += 2;
  return W;
}

// What a warp still has to fetch.  Records are taken in batches of up to 32 of one pair, whose addresses the
// lanes work out once (lane i: record i); units are handed out from the batch.
struct Feed {
  int b, r, tile, n, left;       // the next batch: record `tile` of pair (b, r) (r: kv head * slices + slice) with n; left in the range
  int bb, br, bt, count, pos;    // the batch: its pair, first record and length; the next unit's first record in it
  uint32_t good;                 // bit i: record i's page id is good
  bool starts, ends, closes;     // the batch begins its pair (or the range); it ends its pair; it ends its pair or the range
  const uint8_t* addr;
};

// Up to kUnitTiles consecutive records of one pair.
struct Unit {
  int b, r, tile;
  uint32_t have;                 // bit i: record i's copy was started (its page id is good)
  bool start, ends, last;        // the pair (or range) begins with it; the pair ends with it; the pair or the range does
};

__device__ __forceinline__ int tiles_of(const int* prefix, int b) { return prefix[b + 1] - prefix[b]; }

__device__ __forceinline__ void next_batch(const Q4AttnArgs& a, const int* prefix, int HS, int tpp, Feed& f, int lane) {
  f.starts = f.tile == 0 || f.count == 0;
  f.bb = f.b;
  f.br = f.r;
  f.bt = f.tile;
  f.count = min(min(32, f.n - f.tile), f.left);
  f.pos = 0;
  const int t = f.tile + lane, page = t / tpp, in = t - page * tpp;
  const int id = lane < f.count ? a.page_table[static_cast<size_t>(f.b) * a.max_pages + page] : -1;
  const bool ok = id >= 0 && id < a.num_pages;
  if (lane < f.count && !ok) report(a.status, ZF_DEV_BAD_PAGE_ID);
  f.good = __ballot_sync(0xFFFFFFFFu, ok);
  const int g = a.slices == 1 ? f.r : f.r / a.slices;
  f.addr = a.records + ((static_cast<size_t>(ok ? id : 0) * a.hkv + g) * tpp + in) * kQ4Record;
  f.tile += f.count;
  f.left -= f.count;
  f.ends = f.tile == f.n;
  f.closes = f.ends || f.left == 0;
  if (f.ends && f.left > 0) {                            // the next pair with records
    f.tile = 0;
    if (++f.r == HS) {
      f.r = 0;
      do ++f.b; while (tiles_of(prefix, f.b) == 0);
      f.n = tiles_of(prefix, f.b);
    }
  }
}

// Take the next unit and start its copies into `stage`.
__device__ __forceinline__ Unit next_unit(const Q4AttnArgs& a, const int* prefix, int HS, int tpp, Feed& f,
                                          uint8_t* stage, uint64_t* bar, int lane, uint64_t policy) {
  static_assert(kUnitTiles == 2, "a lane pair holds a unit");
  if (f.pos >= f.count) next_batch(a, prefix, HS, tpp, f, lane);
  Unit u;
  u.b = f.bb;
  u.r = f.br;
  u.tile = f.bt + f.pos;
  u.have = (f.good >> f.pos) & 3u;
  u.start = f.starts && f.pos == 0;
  if (u.have != 0) {
    if (lane == f.pos) mbar_arrive_expect_tx(bar, __popc(u.have) * kQ4Record);
    __syncwarp();
    if ((lane & ~1) == f.pos && (f.good >> lane) & 1u)
      bulk_copy_g2s(stage + (lane & 1) * kQ4Record, f.addr, kQ4Record, bar, policy);
  }
  f.pos += kUnitTiles;
  u.last = f.closes && f.pos >= f.count;
  u.ends = f.ends && f.pos >= f.count;
  return u;
}

// kMulti: several new tokens per request (a causal mask on the last positions).
// kFold (kNT = 1, at most 4 columns): columns 4 to 7 repeat 0 to 3, and in the second product the first
// four carry the weights' high parts and the others the remainders, so that one MMA does the work of two.
template <int kNT, bool kMulti, bool kFold>
__global__ void __launch_bounds__(Q4Cfg<kNT>::kThreads, 1) attn_q4_kernel(const Q4AttnArgs a) {
  using C = Q4Cfg<kNT>;
  constexpr int kWarps = C::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  const Q4Smem L = q4_smem<kNT>(a.batch);
  int* prefix = reinterpret_cast<int*>(smem + L.prefix);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars) + warp * kWarpStages;       // this warp's
  uint8_t* stages = smem + L.stages + static_cast<size_t>(warp) * kWarpStages * kStageQ4;
  uint8_t* qbuf = smem + L.qbuf + static_cast<size_t>(warp) * C::kCols * kQ4QRowBytes;
  Q4Columns<kNT>& cols = reinterpret_cast<Q4Columns<kNT>*>(smem + L.cols)[warp];
  // (tests of the waits: the first stage expects one arrival more, which comes when its wait has run out)
  if (lane < kWarpStages) mbar_init(&bars[lane], a.hold_copies && lane == 0 ? 2 : 1);
  fence_mbar_init();
  wait_prior_grid();          // inputs may come from the preceding grid
  allow_next_grid();

  // ---- records per request and their prefix sums
  const int max_len = a.max_pages * a.page_size;
  for (int b = tid; b < a.batch; b += C::kThreads) {
    int len = a.seq_lens[b];
    if (len < 0 || len > max_len) {
      if (blockIdx.x == 0) report(a.status, ZF_DEV_BAD_SEQ_LEN);
      len = min(max(len, 0), max_len);
    }
    prefix[b + 1] = (len + 15) >> 4;
  }
  if (tid == 0) prefix[0] = 0;
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int base = 0; base < a.batch; base += 32) {
      const int i = base + lane;
      int v = i < a.batch ? prefix[i + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += t;
      }
      if (i < a.batch) prefix[i + 1] = carry + v;
      carry += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
  }
  __syncthreads();
  const int HS = a.hkv * a.slices, tpp = a.page_size >> 4;
  const long long total = static_cast<long long>(HS) * prefix[a.batch];
  const int ranges = gridDim.x * kWarps;
  const int W = range_length(total, ranges, prefix[a.batch] / a.batch);
  if (blockIdx.x == 0) {                                 // for the merge
    for (int b = tid; b <= a.batch; b += C::kThreads) a.prefix[b] = prefix[b];
    if (tid == 0) a.prefix[a.batch + 1] = W;
  }
  // neighbouring ranges go to different SMs: short calls spread over all of them
  const int range = warp * gridDim.x + blockIdx.x;
  const long long lo = static_cast<long long>(range) * W;
  if (lo >= total) return;

  Feed f;
  {
    int l = 0, h = a.batch;                              // the request holding record lo: the largest b with
    while (h - l > 1) {                                  // HS * prefix[b] <= lo that has records
      const int mid = (l + h) >> 1;
      if (static_cast<long long>(HS) * prefix[mid] <= lo) l = mid; else h = mid;
    }
    f.b = l;
    f.n = tiles_of(prefix, l);
    const long long in = lo - static_cast<long long>(HS) * prefix[l];
    f.r = static_cast<int>(in / f.n);
    f.tile = static_cast<int>(in - static_cast<long long>(f.r) * f.n);
    f.left = static_cast<int>(min(static_cast<long long>(W), total - lo));
    f.count = f.pos = 0;
  }
  const uint64_t policy = l2_evict_first_policy();
  const int gi = lane >> 2, ti = lane & 3;
  const int v_lane = kQ4VCodes + 128 * ti + 8 * (gi ^ ((ti & 1) << 2));     // V codes of tokens 2ti (+1, +8, +9)
  const uint8_t* qrow = qbuf + gi * kQ4QRowBytes + 16 * ti;
  constexpr uint32_t kAll = (1u << kUnitTiles) - 1;
  const float fold_c = ti < 2 ? 0.f : 1.f;
  const uint32_t fold_s = ti < 2 ? 0u : 0x80000000u;

  float mx[kNT][2], l[kNT][2];                  // running maximum (rounded up) less kPShift, sum; columns 2ti, 2ti+1
  float cs[kNT][2];                             // kNT = 1: score factor (read per unit otherwise, to spare registers)
  float o[kNT][8][4];
  int len = 0, causal_lim = 0, nh = 0;
  int slot = 0;                                 // partial of the range the current pair would write
  bool whole = false;                           // the current pair began with its first record
  int cb = 0;                                   // its request
  uint32_t phase = 0;                           // bit s: parity of the next wait on stage s
  int sidx = 0;
  Unit u = next_unit(a, prefix, HS, tpp, f, stages, &bars[0], lane, policy);
  while (true) {
    const bool more = f.left > 0 || f.pos < f.count;
    Unit next{};
    // With up to 4 columns, where the copies set the pace, a pair's query rows are staged before the next unit's
    // copies start, so that the range's first unit arrives sooner (ragged workload 68.7 -> 67.2 us, long
    // context 109.4 -> 107.6); with more the copies go first (five to eight columns 127.0 against 127.4).
    if (!kFold && more)
      next = next_unit(a, prefix, HS, tpp, f, stages + (sidx ^ 1) * kStageQ4, &bars[sidx ^ 1], lane, policy);
    if (u.start) {
      whole = u.tile == 0;
      cb = u.b;
      len = min(max(a.seq_lens[u.b], 0), max_len);
      const int g = a.slices == 1 ? u.r : u.r / a.slices;
      const int s = u.r - g * a.slices;
      const int h0 = g * a.group + s * C::kCols;
      nh = min(C::kCols, a.group - s * C::kCols);
      stage_q<kNT, kFold>(a, u.b, h0, nh, qbuf, cols, lane);
      __syncwarp();
      causal_lim = kMulti ? len - a.tokens : 0;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[n][e] = kUnseen;
          l[n][e] = 0.f;
          if (kNT == 1) cs[n][e] = cols.scale[2 * ti + e];
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) o[n][mt][0] = o[n][mt][1] = o[n][mt][2] = o[n][mt][3] = 0.f;
      }
    }
    if (kFold && more)
      next = next_unit(a, prefix, HS, tpp, f, stages + (sidx ^ 1) * kStageQ4, &bars[sidx ^ 1], lane, policy);
    if (u.have) {
      // One outcome for the warp: lanes time their waits on their own, and what follows needs all of them.  (The
      // vote costs the ragged workload 68.3 -> 68.9 us and the long context 109.3 -> 110.6, as much as a bare warp
      // barrier does; taken together with the vote on the scores below, the same and 4% at 14 and 21 columns.)
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars[sidx], (phase >> sidx) & 1u, a.wait_limit_ns))) {
        if (lane == 0) {
          report(a.status, ZF_DEV_TIMEOUT);
          if (a.hold_copies) mbar_arrive(&bars[0]);
        }
        // copies still in flight must land before the CTA exits
        mbar_wait(&bars[sidx], (phase >> sidx) & 1u);
        if (next.have) mbar_wait(&bars[sidx ^ 1], (phase >> (sidx ^ 1)) & 1u);
        return;
      }
      phase ^= 1u << sidx;
      const uint8_t* st = stages + sidx * kStageQ4;
      const int pos0 = 16 * u.tile;                        // position of the unit's first token
      // whether every token counts for every column; if not, ntok[i] tokens of record i do (none of a
      // bad page's)
      const bool full = u.have == kAll && pos0 + 16 * kUnitTiles <= (kMulti ? min(len, causal_lim + 1) : len);
      int ntok[kUnitTiles];
#pragma unroll
      for (int i = 0; i < kUnitTiles; ++i) ntok[i] = 16;
      if (!full) {
#pragma unroll
        for (int i = 0; i < kUnitTiles; ++i) ntok[i] = (u.have >> i) & 1u ? min(16, len - (pos0 + 16 * i)) : 0;
      }

      // ---- S^T (16 tokens x 8 kNT columns) = K (16 x 128) . Q^T, per record
      float x[kNT][kUnitTiles][4];
      uint4 kc[kUnitTiles][2];
      uint32_t ks[kUnitTiles][4];      // scale pairs: (row gi, row gi + 8) x (block 2ti, 2ti + 1)
#pragma unroll
      for (int i = 0; i < kUnitTiles; ++i) {
        const uint8_t* rec = st + i * kQ4Record;
        kc[i][0] = *reinterpret_cast<const uint4*>(rec + 64 * gi + 16 * ti);
        kc[i][1] = *reinterpret_cast<const uint4*>(rec + 64 * (gi + 8) + 16 * ti);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + kQ4KScales + 16 * gi + 4 * ti) & 0x7F7F7F7Fu;
        ks[i][0] = __byte_perm(w, 0u, 0x4040u) << 7;      // token gi, block 2ti
        ks[i][1] = __byte_perm(w, 0u, 0x4242u) << 7;      // token gi + 8, block 2ti
        ks[i][2] = __byte_perm(w, 0u, 0x4141u) << 7;      // token gi, block 2ti + 1
        ks[i][3] = __byte_perm(w, 0u, 0x4343u) << 7;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {    // k-steps 2j and 2j + 1: channels 32 ti + 8 j .. + 7
        uint4 q[kNT];
#pragma unroll
        for (int n = 0; n < kNT; ++n) q[n] = *reinterpret_cast<const uint4*>(qrow + 8 * n * kQ4QRowBytes + 64 * j);
#pragma unroll
        for (int i = 0; i < kUnitTiles; ++i) {
          uint32_t ka[4], kb[4];
          q4_decode4(j == 0 ? kc[i][0].x : j == 1 ? kc[i][0].y : j == 2 ? kc[i][0].z : kc[i][0].w, ka);
          q4_decode4(j == 0 ? kc[i][1].x : j == 1 ? kc[i][1].y : j == 2 ? kc[i][1].z : kc[i][1].w, kb);
          const uint32_t sa = ks[i][j < 2 ? 0 : 2], sb = ks[i][j < 2 ? 1 : 3];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ka[e] = mul_f16x2(ka[e], sa);
            kb[e] = mul_f16x2(kb[e], sb);
          }
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            if (j == 0) mma_f16_zero(x[n][i], ka[0], kb[0], ka[1], kb[1], q[n].x, q[n].y);
            else mma_f16(x[n][i], ka[0], kb[0], ka[1], kb[1], q[n].x, q[n].y);
            mma_f16(x[n][i], ka[2], kb[2], ka[3], kb[3], q[n].z, q[n].w);
          }
        }
      }

      // ---- online softmax, log2 domain.  lane: tokens gi, gi + 8 x columns 2ti, 2ti + 1 (per n).  (Scores are
      // rounded before the maximum comes off: a fused difference would miss the maximum, one of the
      // rounded scores, where floats lie further apart than exponents.)
      bool grow = false;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const F2 f = kNT == 1 ? F2{cs[n][0], cs[n][1]} : F2{cols.scale[8 * n + 2 * ti], cols.scale[8 * n + 2 * ti + 1]};
#pragma unroll
        for (int i = 0; i < kUnitTiles; ++i) {
#pragma unroll
          for (int r = 0; r < 4; r += 2) {
            const F2 y = mul2(F2{x[n][i][r], x[n][i][r + 1]}, f);
            x[n][i][r] = y.x;
            x[n][i][r + 1] = y.y;
          }
        }
      }
      if (!full) {
#pragma unroll
        for (int i = 0; i < kUnitTiles; ++i) {
          const int pos = pos0 + 16 * i + gi;                // this lane's first token; the second is pos + 8
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // (kMulti) the last position that column sees
              const int last = kMulti ? causal_lim + cols.token[8 * n + 2 * ti + e] : INT_MAX;
              if (gi >= ntok[i] || pos > last) x[n][i][e] = -CUDART_INF_F;
              if (gi + 8 >= ntok[i] || pos + 8 > last) x[n][i][e + 2] = -CUDART_INF_F;
            }
          }
        }
      }
      float top[kNT][2];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[n][e] = fmaxf(x[n][0][e], x[n][0][e + 2]);
#pragma unroll
          for (int i = 1; i < kUnitTiles; ++i) top[n][e] = fmaxf(top[n][e], fmaxf(x[n][i][e], x[n][i][e + 2]));
          // (rounded down: the weights fit fp16 however far apart floats lie at the maximum)
          grow |= top[n][e] > __fadd_rd(mx[n][e], kRescaleThreshold + kPShift);
        }
      }
      if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = top[n][e];
#pragma unroll
            for (int dd = 4; dd < 32; dd <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, dd));
            const float mn = fmaxf(mx[n][e], ceilf(v) - kPShift);      // finite: kUnseen at least
            al[e] = fast_exp2(mx[n][e] - mn);
            mx[n][e] = mn;
            l[n][e] *= al[e];
          }
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            o[n][mt][0] *= al[0];
            o[n][mt][1] *= al[1];
            o[n][mt][2] *= al[0];
            o[n][mt][3] *= al[1];
          }
        }
      }

      // P^T as the B operand (k = token, n = column): fp16 high part (the float's first 11 bits) and
      // fp16 remainder (a register pair holds the two columns of a token)
      uint32_t bh[kNT][kUnitTiles][2], bl[kNT][kUnitTiles][2];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
#pragma unroll
        for (int i = 0; i < kUnitTiles; ++i) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const F2 z = add2(F2{x[n][i][2 * r], x[n][i][2 * r + 1]}, F2{-mx[n][0], -mx[n][1]});
            const F2 p = F2{fast_exp2(z.x), fast_exp2(z.y)};
            const F2 sum = add2(F2{l[n][0], l[n][1]}, p);
            l[n][0] = sum.x;
            l[n][1] = sum.y;
            uint32_t hx = __float_as_uint(p.x) & 0xFFFFE000u, hy = __float_as_uint(p.y) & 0xFFFFE000u;
            F2 hi, lo;
            if (kFold) {          // lanes ti < 2: the high part (0 p + h); the others: the remainder (1 p - h)
              hi = fma2(p, F2{fold_c, fold_c}, F2{__uint_as_float(hx ^ fold_s), __uint_as_float(hy ^ fold_s)});
            } else {
              hi = F2{__uint_as_float(hx), __uint_as_float(hy)};
              lo = add2(p, F2{-hi.x, -hi.y});
            }
            bh[n][i][r] = flip8x8(pack_f16x2(hi.x, hi.y));
            if (!kFold) bl[n][i][r] = flip8x8(pack_f16x2(lo.x, lo.y));
          }
        }
      }

      // ---- O^T (128 channels x columns) += V^T (128 x 16 tokens) . P^T.  m-tile mt: row gi is
      // channel 16 gi + 2 mt, row gi + 8 the next one; k: tokens 2ti, 2ti+1, 2ti+8, 2ti+9.
      uint32_t vs[kUnitTiles][2];
      uint2 vw[kUnitTiles][4];
#pragma unroll
      for (int i = 0; i < kUnitTiles; ++i) {
        const uint8_t* rec = st + i * kQ4Record;
        uint32_t w = *reinterpret_cast<const uint32_t*>(rec + kQ4VScales + 16 * gi + 4 * ti) & 0x7F7F7F7Fu;
        if (!full) {              // what lies past the context counts as 0
          w &= (2 * ti < ntok[i] ? 0x000000FFu : 0u) | (2 * ti + 1 < ntok[i] ? 0x0000FF00u : 0u) |
               (2 * ti + 8 < ntok[i] ? 0x00FF0000u : 0u) | (2 * ti + 9 < ntok[i] ? 0xFF000000u : 0u);
        }
        vs[i][0] = __byte_perm(w, 0u, 0x4140u) << 7;
        vs[i][1] = __byte_perm(w, 0u, 0x4342u) << 7;
        vw[i][0] = *reinterpret_cast<const uint2*>(rec + v_lane);
        vw[i][1] = *reinterpret_cast<const uint2*>(rec + v_lane + 64);
        vw[i][2] = *reinterpret_cast<const uint2*>(rec + v_lane + 512);
        vw[i][3] = *reinterpret_cast<const uint2*>(rec + v_lane + 576);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[kUnitTiles][4][4];       // [record][register of the operand][m-tile]
#pragma unroll
        for (int i = 0; i < kUnitTiles; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = h ? vw[i][k].y : vw[i][k].x;
          q4_decode4((w[0] & 0x0F0F0F0Fu) | ((w[1] << 4) & 0xF0F0F0F0u), v[i][0]);
          q4_decode4(((w[0] >> 4) & 0x0F0F0F0Fu) | (w[1] & 0xF0F0F0F0u), v[i][1]);
          q4_decode4((w[2] & 0x0F0F0F0Fu) | ((w[3] << 4) & 0xF0F0F0F0u), v[i][2]);
          q4_decode4(((w[2] >> 4) & 0x0F0F0F0Fu) | (w[3] & 0xF0F0F0F0u), v[i][3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[i][0][e] = mul_f16x2(v[i][0][e], vs[i][0]);
            v[i][1][e] = mul_f16x2(v[i][1][e], vs[i][0]);
            v[i][2][e] = mul_f16x2(v[i][2][e], vs[i][1]);
            v[i][3][e] = mul_f16x2(v[i][3][e], vs[i][1]);
          }
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float s[4];
            mma_f16_zero(s, v[0][0][e], v[0][1][e], v[0][2][e], v[0][3][e], bh[n][0][0], bh[n][0][1]);
#pragma unroll
            for (int i = 1; i < kUnitTiles; ++i)
              mma_f16(s, v[i][0][e], v[i][1][e], v[i][2][e], v[i][3][e], bh[n][i][0], bh[n][i][1]);
            if (!kFold) {
#pragma unroll
              for (int i = 0; i < kUnitTiles; ++i)
                mma_f16(s, v[i][0][e], v[i][1][e], v[i][2][e], v[i][3][e], bl[n][i][0], bl[n][i][1]);
            }
            add4(o[n][4 * h + e], s);
          }
        }
      }
    }
    if (u.last) {
      // ---- the pair, or the range, ends: its result or a partial.  A lane holds 16 consecutive channels
      // of two columns (of one, when columns are folded: the halves of a column's sum meet first).
      const bool done = whole && u.ends;
      const size_t part = (static_cast<size_t>(range) * 2 + slot) * C::kCols;
      slot = 1;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        // this lane's 16 channels of column col of the tile, from x[channel]; m, s: its maximum and sum
        auto put = [&](int col, float m, float s, const float (&x)[16]) {
          if (col >= nh) return;
          float* dst;
          float f = 1.f;
          if (done) {
            const size_t row = static_cast<size_t>(cb) * a.hq + cols.at[col];
            dst = a.out + row * ZF_HEAD_DIM;
            f = s == 0.f ? 0.f : a.v_factor / s;           // a sum of 0: nothing was seen; a NaN sum stays a NaN
            if (gi == 0) a.lse[row] = s == 0.f ? -CUDART_INF_F : (m + log2f(s)) * kLn2;
          } else {
            dst = a.part_o + (part + col) * ZF_HEAD_DIM;
            if (gi == 0) a.part_ml[part + col] = make_float2(m, s);
          }
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<float4*>(dst + 16 * gi + k) = make_float4(x[k] * f, x[k + 1] * f, x[k + 2] * f, x[k + 3] * f);
        };
        float x[2][16];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int dd = 4; dd < 32; dd <<= 1) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], dd);
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            x[e][2 * mt] = o[n][mt][e];
            x[e][2 * mt + 1] = o[n][mt][2 + e];
          }
        }
        if (kFold) {              // lanes ti < 2 take column 2 ti, the others column 2 (ti - 2) + 1
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float mine = ti < 2 ? x[0][i] : x[1][i], other = ti < 2 ? x[1][i] : x[0][i];
            x[0][i] = mine + __shfl_xor_sync(0xFFFFFFFFu, other, 2);
          }
          put(ti < 2 ? 2 * ti : 2 * (ti - 2) + 1, ti < 2 ? mx[n][0] : mx[n][1], ti < 2 ? l[n][0] : l[n][1], x[0]);
        } else {
          put(8 * n + 2 * ti, mx[n][0], l[n][0], x[0]);
          put(8 * n + 2 * ti + 1, mx[n][1], l[n][1], x[1]);
        }
      }
    }
    __syncwarp();                // the stage, and at a pair's end the query rows, may be overwritten
    if (!more) break;
    u = next;
    sidx ^= 1;
  }
}

// The merge: kPerRow warps per (request, query head, new token) take turns at its partials.  A partial holds its weighted sum of values as it is, its maximum and its sum; the maxima are whole
// numbers, so the partials' factors are powers of two and the merge adds no rounding but those of its
// sums (a log-sum-exp near 20, kept as one float, would be off by 2^-20 in each weight).  Rows whose
// pair lies in one range were finished by the attention kernel.
struct Q4MergeArgs {
  const float* part_o;
  const float2* part_ml;
  const int32_t* prefix;
  float* out;
  float* lse;
  int32_t batch, hq, group, slices, tokens, cols;
  float v_factor;
};
constexpr int kMergePre = 8;                     // partials a warp reads at once
constexpr int kMergeOne = 16, kMergeFour = 48;    // up to so many partials: one or four warps per row
template <int kPerRow>
constexpr int kMergeRows = kPerRow < 4 ? 4 / kPerRow : 1;          // rows per CTA
template <int kPerRow>
__global__ void __launch_bounds__(kMergeRows<kPerRow> * kPerRow * 32) q4_merge_kernel(const Q4MergeArgs a) {
  constexpr int kRows = kMergeRows<kPerRow>;
  __shared__ float4 sh_o[kRows * kPerRow][32];
  __shared__ float2 sh_ml[kRows * kPerRow];
  const int lane = threadIdx.x & 31;
  const int all = threadIdx.x >> 5, warp = all % kPerRow, base = all - warp;      // warp: among the row's
  const int idx = blockIdx.x * kRows + all / kPerRow;
  const bool in = idx < a.batch * a.hq;
  const int b = in ? idx / a.hq : 0, h = in ? idx - b * a.hq : 0;
  const int g = h / a.group, hg = h - g * a.group;
  const int s = hg / a.cols, col = hg - s * a.cols;
  allow_next_grid();
  wait_prior_grid();
  const int p0 = a.prefix[b], n = a.prefix[b + 1] - p0, W = a.prefix[a.batch + 1];
  const size_t row = query_row(b, h, a.tokens, a.hq);
  if (in && n == 0) {                            // an empty request
    if (warp == 0) *reinterpret_cast<float4*>(a.out + row * ZF_HEAD_DIM + 4 * lane) = make_float4(0.f, 0.f, 0.f, 0.f);
    if (warp == 0 && lane == 0) a.lse[row] = -CUDART_INF_F;
  }
  const int HS = a.hq / a.group * a.slices;
  const long long S = static_cast<long long>(HS) * p0 + static_cast<long long>(g * a.slices + s) * n;
  int k0 = 0, k1 = 0;
  if (in && n > 0) {
    k0 = static_cast<int>(S / W);
    k1 = static_cast<int>((S + n - 1) / W);
  }
  if (k0 == k1 && kRows == 1) return;            // (the warps of other rows of the CTA meet at a barrier below)
  const bool live = k0 != k1;
  // range k's partial of this pair: its first, unless the pair began within range k0
  const int first = S == static_cast<long long>(k0) * W ? 0 : 1;
  auto at = [&](int k) { return (static_cast<size_t>(k) * 2 + (k == k0 ? first : 0)) * a.cols + col; };
  float M = kUnseen, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = k0 + warp; live && k <= k1; k += kPerRow * kMergePre) {
    float2 ml[kMergePre];
    float4 v[kMergePre];
#pragma unroll
    for (int j = 0; j < kMergePre; ++j) {
      const int kk = k + j * kPerRow;
      ml[j] = make_float2(kUnseen, 0.f);
      v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (kk <= k1) {
        ml[j] = a.part_ml[at(kk)];
        v[j] = reinterpret_cast<const float4*>(a.part_o + at(kk) * ZF_HEAD_DIM)[lane];
      }
    }
    float top = M;
#pragma unroll
    for (int j = 0; j < kMergePre; ++j) top = fmaxf(top, ml[j].x);
    const float f0 = fast_exp2(M - top);
    M = top;
    sum *= f0;
    acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
#pragma unroll
    for (int j = 0; j < kMergePre; ++j) {
      const float f = fast_exp2(ml[j].x - M);
      sum += f * ml[j].y;
      acc.x += f * v[j].x;
      acc.y += f * v[j].y;
      acc.z += f * v[j].z;
      acc.w += f * v[j].w;
    }
  }
  if (kPerRow > 1) {
    sh_o[all][lane] = acc;
    if (lane == 0) sh_ml[all] = make_float2(M, sum);
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < kPerRow; ++w) M = fmaxf(M, sh_ml[base + w].x);
    sum = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kPerRow; ++w) {
      const float f = fast_exp2(sh_ml[base + w].x - M);
      sum += f * sh_ml[base + w].y;
      const float4 v = sh_o[base + w][lane];
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
  }
  if (!live) return;
  const float inv = sum == 0.f ? 0.f : a.v_factor / sum;           // a NaN sum stays a NaN
  *reinterpret_cast<float4*>(a.out + row * ZF_HEAD_DIM + 4 * lane) =
      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (lane == 0) a.lse[row] = sum == 0.f ? -CUDART_INF_F : (M + log2f(sum)) * kLn2;
}

// Passes over a kv head's records (slices) and 8-column tiles per pass (1 to 4): as few passes as hold the
// columns, of equal width.  Wider passes decode each record once for more columns.  Measured at 32 requests
// of 8192 tokens: 28/4 heads, two new tokens (14 columns) 57.2 us in one pass of two tiles, 71.1 in two of
// one; three (21) 77.8 in one of three, 93.8 in one of four, 96.9 in two of two; four (28) 94.8 in one of
// four, 97.9 in two of two, 127.9 in four of one.  32/8 heads, five new tokens (20) 139.8 in one of three,
// 171.5 in one of four.
int q4_slices(int cols) { return (cols + 31) / 32; }
int q4_col_tiles(int cols) {
  const int tiles = (cols + 7) / 8, slices = q4_slices(cols);
  return (tiles + slices - 1) / slices;
}
static_assert(Q4Cfg<3>::kWarps == Q4Cfg<4>::kWarps);
int q4_warps(int nt) { return nt == 1 ? Q4Cfg<1>::kWarps : nt == 2 ? Q4Cfg<2>::kWarps : Q4Cfg<4>::kWarps; }

// Grid and workspace: two partials per range, whatever the lengths; the prefix sums of the records.
struct Q4Plan {
  int nt = 1, slices = 1, grid = 1;
  size_t o_bytes = 0, ml_bytes = 0, prefix_bytes = 0;
  size_t bytes() const { return o_bytes + ml_bytes + prefix_bytes; }
};
Q4Plan q4_plan(int batch, int hq, int hkv, int page_size, int max_pages, int sms) {
  Q4Plan p;
  const int group = hq / hkv;
  p.nt = q4_col_tiles(group);
  p.slices = q4_slices(group);
  const long long most = static_cast<long long>(batch) * hkv * p.slices * max_pages * (page_size / 16);
  const long long units = (most + kUnitTiles - 1) / kUnitTiles;
  p.grid = static_cast<int>(units < sms ? (units > 0 ? units : 1) : sms);
  // (several passes count as passes of 32, so that more tokens never need a smaller workspace)
  const int width = p.slices > 1 ? 4 : p.nt;
  const size_t parts = static_cast<size_t>(p.grid) * q4_warps(p.nt) * 2 * 8 * width;
  p.o_bytes = parts * ZF_HEAD_DIM * 4;
  p.ml_bytes = parts * 8;
  p.prefix_bytes = ((static_cast<size_t>(batch) + 2) * 4 + 255) & ~static_cast<size_t>(255);
  return p;
}

template <typename Kernel, typename Args>
zf_status launch_pdl(Kernel kernel, int grid, int threads, size_t smem, cudaStream_t s, const Args& args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess ? ZF_OK : ZF_ERR_CUDA;
}

template <int kNT, bool kMulti, bool kFold = false>
zf_status launch_q4(const Q4AttnArgs& a, int grid, int which, cudaStream_t s) {
  const size_t smem = q4_smem<kNT>(a.batch).total;
  const zf_status st = ensure_smem_limit(reinterpret_cast<const void*>(attn_q4_kernel<kNT, kMulti, kFold>), which, smem);
  if (st != ZF_OK) return st;
  return launch_pdl(attn_q4_kernel<kNT, kMulti, kFold>, grid, Q4Cfg<kNT>::kThreads, smem, s, a);
}

}  // namespace

static bool q4_shape_ok(int32_t batch, int32_t tokens, int32_t hq, int32_t hkv, int32_t max_pages) {
  return tokens_ok(tokens, hq) && attn_shape_ok(batch, hq, hkv, max_pages) &&
         attn_shape_ok(batch, hq * tokens, hkv, max_pages);
}

}  // namespace zf

using namespace zf;

extern "C" size_t zf_q4_decode_attn_workspace_size(int32_t batch, int32_t tokens, int32_t num_q_heads,
                                                   int32_t num_kv_heads, int32_t page_size,
                                                   int32_t max_pages_per_req) {
  if (!q4_shape_ok(batch, tokens, num_q_heads, num_kv_heads, max_pages_per_req)) return 0;
  if (page_size < ZF_BLOCK_TOKENS || page_size % ZF_BLOCK_TOKENS || page_size > ZF_MAX_PAGE_SIZE) return 0;
  int sms = 0;
  if (current_sm_count(&sms) != ZF_OK) return 0;
  return q4_plan(batch, num_q_heads * tokens, num_kv_heads, page_size, max_pages_per_req, sms).bytes();
}

static zf_status q4_decode_attn(const zf_q4_cache* c, const uint16_t* q, int32_t batch, int32_t tokens,
                                int32_t num_q_heads, const int32_t* page_table, int32_t max_pages,
                                const int32_t* seq_lens, float softmax_scale, float* out, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream, uint64_t wait_limit_ns = kWaitTimeoutNs,
                                bool hold_copies = false) {
  zf_status st = check_q4_cache(c);
  if (st != ZF_OK) return st;
  if (!q4_shape_ok(batch, tokens, num_q_heads, c->num_kv_heads, max_pages)) return ZF_ERR_INVALID_ARGUMENT;
  if (batch == 0) return ZF_OK;
  if (!q || !page_table || !seq_lens || !out || !lse || !workspace) return ZF_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(page_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return ZF_ERR_INVALID_ARGUMENT;
  // the scores' factor, with the cache's scale and the scale decoding's 2^-8 in it, must be a float
  const float scale_log2 = softmax_scale * c->k_scale * (1.4426950408889634f * kQ4ScaleFactor);
  if (!(scale_log2 >= -1e37f && scale_log2 <= 1e37f)) return ZF_ERR_INVALID_ARGUMENT;
  // the records of all requests are counted with 32 bits
  if (static_cast<long long>(batch) * max_pages * (c->page_size / 16) > INT_MAX) return ZF_ERR_UNSUPPORTED;
  int sms = 0;
  if ((st = current_sm_count(&sms)) != ZF_OK) return st;
  const int32_t hq = num_q_heads * tokens;
  const Q4Plan p = q4_plan(batch, hq, c->num_kv_heads, c->page_size, max_pages, sms);
  if (workspace_bytes < p.bytes()) return ZF_ERR_WORKSPACE_TOO_SMALL;

  Q4AttnArgs a{};
  a.records = c->records;
  a.status = c->status;
  a.q = q;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.o_bytes);
  a.prefix = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + p.o_bytes + p.ml_bytes);
  a.batch = batch;
  a.hq = hq;
  a.hkv = c->num_kv_heads;
  a.group = hq / c->num_kv_heads;
  a.tokens = tokens;
  a.slices = p.slices;
  a.page_size = c->page_size;
  a.num_pages = c->num_pages;
  a.max_pages = max_pages;
  a.scale_log2 = scale_log2;
  a.v_factor = c->v_scale * kQ4ScaleFactor;
  a.wait_limit_ns = wait_limit_ns;
  a.hold_copies = hold_copies;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool multi = tokens > 1;
  if (a.group <= 4) st = multi ? launch_q4<1, true, true>(a, p.grid, 4, s) : launch_q4<1, false, true>(a, p.grid, 5, s);
  else if (p.nt == 1) st = multi ? launch_q4<1, true>(a, p.grid, 0, s) : launch_q4<1, false>(a, p.grid, 1, s);
  else if (p.nt == 2) st = launch_q4<2, true>(a, p.grid, 2, s);
  else if (p.nt == 3) st = launch_q4<3, true>(a, p.grid, 6, s);
  else st = launch_q4<4, true>(a, p.grid, 3, s);
  if (st != ZF_OK) return st;

  Q4MergeArgs m{};
  m.part_o = a.part_o;
  m.part_ml = a.part_ml;
  m.prefix = a.prefix;
  m.out = out;
  m.lse = lse;
  m.batch = batch;
  m.hq = hq;
  m.group = a.group;
  m.slices = a.slices;
  m.tokens = tokens;
  m.cols = 8 * p.nt;
  m.v_factor = a.v_factor;
  // warps per row by the partials that a pair of the largest length has (one warp reads kMergePre at once)
  const int rows = batch * hq, most = max_pages * (c->page_size / 16);
  const long long total = static_cast<long long>(batch) * c->num_kv_heads * p.slices * most;
  const int parts = most / range_length(total, p.grid * q4_warps(p.nt), most) + 1;
  if (parts <= kMergeOne) return launch_pdl(q4_merge_kernel<1>, (rows + 3) / 4, 128, 0, s, m);
  if (parts <= kMergeFour) return launch_pdl(q4_merge_kernel<4>, rows, 128, 0, s, m);
  return launch_pdl(q4_merge_kernel<16>, rows, 512, 0, s, m);
}

extern "C" zf_status zf_q4_decode_attn(const zf_q4_cache* cache, const uint16_t* q, int32_t batch, int32_t tokens,
                                       int32_t num_q_heads, const int32_t* page_table, int32_t max_pages_per_req,
                                       const int32_t* seq_lens, float softmax_scale, float* out, float* lse,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  return q4_decode_attn(cache, q, batch, tokens, num_q_heads, page_table, max_pages_per_req, seq_lens, softmax_scale, out,
                        lse, workspace, workspace_bytes, stream);
}

extern "C" zf_status zf_q4_decode_attn_wait_test(const zf_q4_cache* cache, const uint16_t* q, int32_t batch,
                                                 int32_t tokens, int32_t num_q_heads, const int32_t* page_table,
                                                 int32_t max_pages_per_req, const int32_t* seq_lens,
                                                 float softmax_scale, float* out, float* lse, void* workspace,
                                                 size_t workspace_bytes, uint64_t wait_limit_ns, void* stream) {
  if (wait_limit_ns < 1000 || wait_limit_ns > kWaitTimeoutNs) return ZF_ERR_INVALID_ARGUMENT;
  return q4_decode_attn(cache, q, batch, tokens, num_q_heads, page_table, max_pages_per_req, seq_lens, softmax_scale, out,
                        lse, workspace, workspace_bytes, stream, wait_limit_ns, true);
}
