// zf_q4_decode_attn: split-KV decode attention over the 4-bit paged cache (one or several new tokens
// per request), and its split-result merge.
//
// Mathematics.  K and V are code * s (16-channel blocks, e2m1 codes of two significant bits, e4m3
// scales of four): every product code * s has at most six significant bits and is exact in fp16, so
// the operands of the matrix instructions are the stored values themselves.  q (BF16) is brought into
// fp16 by a power of two per row, which its scores take back: exact down to 2^-36 of the row's
// largest value.  Scores, running maximum and sum and the output are float32.  The softmax weights p
// (times 2^7, so that the remainder of a small weight stays clear of fp16's subnormals) are split
// into an fp16 high part and an fp16 remainder, two MMAs: about 22 bits.
//
// Structure: as the attention kernels over the other caches (zf_attn.cu): one persistent CTA per SM,
// the same work split (balanced page ranges, or fixed chunks), a metadata warp one item ahead,
// consumer warps that each stream their own units of kUnitTiles 16-token records into two private
// stages, and a combine of the warps' states at the end of an item.
//  * A record holds K and V of 16 tokens of one kv head: one bulk copy (2304 bytes).
//  * K^T: a lane's A fragments of all eight k-steps are 16 contiguous bytes of a token's row (the order
//    of channels within the k-steps is free as long as q follows it), two 16-byte reads per record, and
//    it meets two scale blocks per token, four scale bytes in one 4-byte read.
//  * V: a lane's rows are the 16 channels of one block (eight m-tiles x two rows), so it needs one scale
//    per token: four tokens' codes in four 8-byte reads, their scales in one 4-byte read.  The codes
//    of two tokens are interleaved by nibble, so that one conversion gives a register of the
//    operand (two tokens, one channel).
//  * e2m1 pairs become half pairs in one conversion, and one multiplication applies the scale.
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
constexpr int kQ4QRowBytes = 320;                        // q row in shared memory (see q_at)
constexpr int kItemTilesQ4 = 2048;                       // records (and pages) of the largest item
constexpr float kPShift = 7.f;                           // weights are 2^7 times their usual size
static_assert(kStageQ4 >= (8 * kOStride + 16) * 4, "a stage holds a warp's combine state of 8 columns");

// Consumer warps by the number of 8-column tiles of a pass (kNT), from the registers they need.
template <int kNT>
struct Q4Cfg {
  static constexpr int kWarps = kNT == 1 ? 15 : kNT == 2 ? 11 : 7;
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kCols = 8 * kNT;
};

struct Q4Smem {
  size_t stages, item_full, q_full, item_empty, misc, desc, meta, qbuf, qscale, bars, prefix, lens, total;
};

template <int kNT>
__host__ __device__ inline Q4Smem q4_smem(int batch) {
  using C = Q4Cfg<kNT>;
  Q4Smem s;
  size_t at = 0;
  s.stages = at; at += static_cast<size_t>(C::kWarps) * kWarpStages * kStageQ4;
  s.item_full = at; at += 2 * 8;
  s.q_full = at; at += 2 * 8;
  s.item_empty = at; at += 2 * 8;
  s.misc = at; at += 16 + 16 * 4;               // [0] abort flag, [16..] combine stage per warp
  s.desc = at; at += 2 * 64;
  s.meta = at; at += 2 * kItemTilesQ4 * 4;
  s.qbuf = at; at += 2 * C::kCols * kQ4QRowBytes;
  s.qscale = at; at += 2 * C::kCols * 4;
  s.bars = at; at += static_cast<size_t>(C::kWarps) * kWarpStages * 8;
  s.prefix = at; at += static_cast<size_t>(batch + 1) * 4;
  s.lens = at; at += static_cast<size_t>(batch) * 4;
  s.total = (at + 127) & ~static_cast<size_t>(127);
  return s;
}

template <int kWarps>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
}

// Barrier over the consumer warps that also ORs a predicate across them.
template <int kWarps>
__device__ __forceinline__ bool consumers_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "n"(kWarps * 32)
      : "memory");
  return r != 0;
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

// d += s, rounded to nearest.  The matrix instructions cut their float sums off instead, a bias that
// grows along a chain of accumulations, so a chain is one unit long and is added to the output here: error
// against 64 bits at the long-context workload 6.1e-7 instead of 2.1e-6, for 2 to 8% of the time.
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

constexpr uint32_t kNoRecord = 0xFFFFFFFFu;

// The item's records into rec[u] (index into the cache, kNoRecord for a bad page), by all 32 lanes.
__device__ __forceinline__ void resolve_records(const AttnArgs& a, const ItemDesc& d, uint32_t* rec, int lane) {
  const int tpp = a.page_size >> 4;
  const int32_t* row = a.page_table + static_cast<size_t>(d.b) * a.max_pages + d.pg0;
  constexpr int kAhead = 8;            // page-table entries per lane read at once
  for (int i0 = lane; i0 < d.npg; i0 += 32 * kAhead) {
    int pid[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) pid[k] = i0 + 32 * k < d.npg ? row[i0 + 32 * k] : -1;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + 32 * k;
      if (i >= d.npg) break;
      const bool ok = pid[k] >= 0 && pid[k] < a.num_pages;
      if (!ok) report(a.status, ZF_DEV_BAD_PAGE_ID);
      const uint32_t first = (static_cast<uint32_t>(pid[k]) * a.hkv + d.g) * tpp;
      for (int t = 0; t < tpp; ++t)
        if (i * tpp + t < d.units) rec[i * tpp + t] = ok ? first + t : kNoRecord;
    }
  }
}

// Start the copies of unit u (records u * kUnitTiles ..) of an item: lane i issues record i's.  Returns
// which records were started (bit i).
__device__ __forceinline__ uint32_t issue_unit(const uint8_t* records, const uint32_t* rec, int units, int u,
                                               uint8_t* stage, uint64_t* bar, int lane, uint64_t policy) {
  const int t = u * kUnitTiles + lane;
  uint32_t r = kNoRecord;
  if (lane < kUnitTiles && t < units) r = rec[t];
  const uint32_t mask = __ballot_sync(0xFFFFFFFFu, r != kNoRecord);
  if (mask == 0) return 0;
  if (lane == 0) mbar_arrive_expect_tx(bar, __popc(mask) * kQ4Record);
  __syncwarp();
  if (r != kNoRecord)
    bulk_copy_g2s(stage + lane * kQ4Record, records + static_cast<size_t>(r) * kQ4Record, kQ4Record, bar, policy);
  return mask;
}

// One q row of 128 BF16 values (lane holds words lane and lane + 32) into shared memory as fp16 times
// a power of two that brings its largest exponent to 11; returns the inverse factor.  Channel c =
// 32 t + 8 j + e goes to byte 64 j + 16 t + 2 e: lane t's words of k-steps 2j, 2j+1 are 16 bytes,
// and the rows' stride spreads a warp's reads over the banks.
__device__ __forceinline__ float store_q_row(uint8_t* row, int lane, uint32_t w0, uint32_t w1, bool negate) {
  const uint32_t m0 = w0 & 0x7FFF7FFFu, m1 = w1 & 0x7FFF7FFFu;
  const uint32_t big = max(max(m0 & 0xFFFFu, m0 >> 16), max(m1 & 0xFFFFu, m1 >> 16));
  const int e = static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, big) >> 7);        // biased exponent
  const int k = min(138 - e, 126);
  const float f = __int_as_float(((127 + k) << 23) | (negate ? 0x80000000 : 0));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w = h ? w1 : w0;
    const int c = 2 * (lane + 32 * h);
    const int t = c >> 5, j = (c >> 3) & 3, r = c & 7;
    *reinterpret_cast<uint32_t*>(row + 64 * j + 16 * t + 2 * r) = pack_f16x2(bf16lo_to_f32(w) * f, bf16hi_to_f32(w) * f);
  }
  return __int_as_float((127 - k) << 23);
}

template <int kNT, bool kFold>
__device__ __forceinline__ void stage_q(const AttnArgs& a, const ItemDesc& d, uint8_t* qb, float* qs, int lane) {
  constexpr int kCols = Q4Cfg<kNT>::kCols;
#pragma unroll
  for (int r0 = 0; r0 < kCols; r0 += 8) {
    uint32_t v[8][2];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int c = kFold ? r & 3 : r0 + r;
      const int qh = d.h0 + min(c, d.nh - 1);
      const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + query_row(d.b, qh, a.tokens, a.hq) * ZF_HEAD_DIM);
      v[r][0] = c < d.nh ? src[lane] : 0u;
      v[r][1] = c < d.nh ? src[lane + 32] : 0u;
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float inv = store_q_row(qb + (r0 + r) * kQ4QRowBytes, lane, v[r][0], v[r][1], a.scale_log2 < 0.f);
      // positive, so that the largest raw score has the largest score, and -inf stays one
      if (lane == 0) qs[r0 + r] = fmaxf(inv * fabsf(a.scale_log2), 1e-37f);
    }
  }
}

// A row's result from its weighted sum of values (lane: channels 4 lane ..), its maximum M and its sum.
// A sum of 0: nothing was seen; a NaN sum stays a NaN.
__device__ __forceinline__ void finish_row(float* out, float* lse, size_t row, int lane, float4 acc, float M, float sum,
                                           float v_factor) {
  const float inv = sum == 0.f ? 0.f : v_factor / sum;
  *reinterpret_cast<float4*>(out + row * ZF_HEAD_DIM + 4 * lane) =
      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (lane == 0) lse[row] = sum == 0.f ? -CUDART_INF_F : (M + log2f(sum)) * kLn2;
}

// kMulti: several new tokens per request (a causal mask on the last positions).
// kFold (kNT = 1, at most 4 columns): columns 4 to 7 repeat 0 to 3, and in the second product the first
// four carry the weights' high parts and the others the remainders, so that one MMA does the work of two.
template <int kNT, bool kMulti, bool kFold>
__global__ void __launch_bounds__(Q4Cfg<kNT>::kThreads, 1) attn_q4_kernel(const AttnArgs a, const float v_factor) {
  using C = Q4Cfg<kNT>;
  constexpr int kWarps = C::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  const Q4Smem L = q4_smem<kNT>(a.batch);
  uint64_t* item_full = reinterpret_cast<uint64_t*>(smem + L.item_full);
  uint64_t* item_empty = reinterpret_cast<uint64_t*>(smem + L.item_empty);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L.q_full);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L.misc);
  int* combine_stage = reinterpret_cast<int*>(smem + L.misc + 16);
  ItemDesc* desc = reinterpret_cast<ItemDesc*>(smem + L.desc);
  uint32_t* meta = reinterpret_cast<uint32_t*>(smem + L.meta);
  uint8_t* qbuf = smem + L.qbuf;
  float* qscale = reinterpret_cast<float*>(smem + L.qscale);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
  int* prefix = reinterpret_cast<int*>(smem + L.prefix);
  int* lens = reinterpret_cast<int*>(smem + L.lens);
  uint8_t* stages = smem + L.stages;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < 2) {
    mbar_init(&item_full[tid], 1);
    mbar_init(&q_full[tid], 1);
    mbar_init(&item_empty[tid], kWarps);
  }
  if (tid < kWarps * kWarpStages) mbar_init(&bars[tid], 1);
  if (tid == 0) *abort_flag = 0;
  fence_mbar_init();
  const int HS = a.hkv * a.slices;
  wait_prior_grid();          // inputs may come from the preceding grid
  allow_next_grid();
  const uint64_t policy = l2_evict_first_policy();
  load_lengths<false, C::kThreads>(a, prefix, lens, tid);       // ends with a barrier (also for the barriers above)
  const Ranges g = make_ranges<kItemTilesQ4, kItemTilesQ4>(a, HS * prefix[a.batch]);

  if (warp == kWarps) {
    // ============================================================== metadata warp
    int k = 0;
    if (a.publish_delay_ns) sleep_for_ns(a.publish_delay_ns);
    auto publish = [&](const ItemDesc& d) -> bool {
      const int buf = k & 1;
      bool good = true;
      if (lane == 0) good = !*abort_flag && mbar_wait(&item_empty[buf], ((k >> 1) & 1u) ^ 1u);
      good = __shfl_sync(0xFFFFFFFFu, good, 0);
      if (!good) {
        if (lane == 0) {
          report(a.status, ZF_DEV_TIMEOUT);
          *abort_flag = 1;
        }
        return false;
      }
      if (d.b >= 0) resolve_records(a, d, meta + buf * kItemTilesQ4, lane);
      __syncwarp();
      if (lane == 0) {
        desc[buf] = d;
        mbar_arrive(&item_full[buf]);        // release: the records can be fetched
      }
      if (d.b >= 0) {
        stage_q<kNT, kFold>(a, d, qbuf + buf * C::kCols * kQ4QRowBytes, qscale + buf * C::kCols, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[buf]);   // release: the q rows
      }
      ++k;
      return true;
    };
    if (walk_range(a, prefix, lens, g, HS, publish)) {
      ItemDesc end_marker{};
      end_marker.b = -1;
      publish(end_marker);
    }
    return;
  }

  // ================================================================== consumer warps
  // partials per pair, for the merge kernel (spread over all CTAs)
  for (int p = blockIdx.x * (kWarps * 32) + tid; p < a.batch * HS; p += gridDim.x * (kWarps * 32)) {
    const int b = p / HS, r = p - b * HS;
    const int n = prefix[b + 1] - prefix[b];
    a.chunk_counts[p] = a.chunk_pages > 0 ? n : n > 0 ? pair_chunks(g, HS * prefix[b] + r * n, n) : 0;
  }
  const int gi = lane >> 2, ti = lane & 3;
  uint8_t* my_stages = stages + static_cast<size_t>(warp) * kWarpStages * kStageQ4;
  uint64_t* my_bars = bars + warp * kWarpStages;
  const int v_lane = kQ4VCodes + 128 * ti + 8 * (gi ^ ((ti & 1) << 2));     // V codes of tokens 2ti (+1, +8, +9)
  uint32_t inflight = 0;        // per stage s, bits (s * kUnitTiles ..): records whose copies are under way
  constexpr uint32_t kAll = (1u << kUnitTiles) - 1;
  bool prefetched = false;      // this warp's first unit of the current item is already in flight
  bool aborted = false;
  int sidx = 0;
  uint32_t phase = 0;
  auto give_up = [&]() {
    aborted = true;
    *abort_flag = 1;
    report(a.status, ZF_DEV_TIMEOUT);
  };
  for (int k = 0;; ++k) {
    const int buf = k & 1;
    if (!aborted && (*abort_flag || !mbar_wait(&item_full[buf], (k >> 1) & 1u, a.wait_limit_ns))) give_up();
    // one decision for all consumer warps: stop at the end marker, or once any wait gave up
    if (consumers_any<kWarps>(aborted || desc[buf].b < 0)) break;
    const ItemDesc d = desc[buf];
    const uint32_t* m = meta + buf * kItemTilesQ4;
    const int nu = (d.units + kUnitTiles - 1) / kUnitTiles;
    const uint8_t* qrow = qbuf + (buf * C::kCols + gi) * kQ4QRowBytes + 16 * ti;

    float mx[kNT][2], l[kNT][2], cs[kNT][2];      // running maximum (rounded up) less kPShift, sum, score factor; columns 2ti, 2ti+1
    int seen[kNT][2];                             // kMulti: last position those columns see
    float o[kNT][8][4];
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[n][e] = kNoScore;
        l[n][e] = 0.f;
        seen[n][e] = kMulti ? lens[d.b] - a.tokens + (d.h0 + (kFold ? (2 * ti + e) & 3 : 8 * n + 2 * ti + e)) % a.tokens : 0;
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) o[n][mt][0] = o[n][mt][1] = o[n][mt][2] = o[n][mt][3] = 0.f;
    }
    const int causal_lim = kMulti ? lens[d.b] - a.tokens : 0;

    if (!prefetched && warp < nu)
      inflight |= issue_unit(a.k_comp, m, d.units, warp, my_stages + sidx * kStageQ4, &my_bars[sidx], lane, policy)
                  << (sidx * kUnitTiles);
    prefetched = false;
    if (!aborted && (*abort_flag || !mbar_wait(&q_full[buf], (k >> 1) & 1u, a.wait_limit_ns))) give_up();
    if (!aborted) {
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) cs[n][e] = qscale[buf * C::kCols + 8 * n + 2 * ti + e];
    }

    for (int u = warp; u < nu && !aborted; u += kWarps) {
      // start the warp's next unit: of this item, or its first one of the next item
      const int un = u + kWarps;
      const int ns = sidx ^ 1;
      uint8_t* next_stage = my_stages + ns * kStageQ4;
      if (un < nu) {
        inflight |= issue_unit(a.k_comp, m, d.units, un, next_stage, &my_bars[ns], lane, policy) << (ns * kUnitTiles);
      } else {
        const int nb = buf ^ 1;       // the next item (or the end marker) is published after this one
        if (*abort_flag || !mbar_wait(&item_full[nb], ((k + 1) >> 1) & 1u, a.wait_limit_ns)) {
          give_up();
          break;
        } else if (desc[nb].b >= 0 && warp < (desc[nb].units + kUnitTiles - 1) / kUnitTiles) {
          inflight |= issue_unit(a.k_comp, meta + nb * kItemTilesQ4, desc[nb].units, warp, next_stage, &my_bars[ns], lane,
                                 policy)
                      << (ns * kUnitTiles);
          prefetched = true;
        }
      }
      // wait for the current unit (nothing armed: all its pages are bad, and it is skipped)
      const uint32_t here = (inflight >> (sidx * kUnitTiles)) & kAll;
      if (here) {
        if (*abort_flag || !mbar_wait(&my_bars[sidx], (phase >> sidx) & 1u)) {
          give_up();
          break;
        }
        phase ^= 1u << sidx;
        inflight &= ~(kAll << (sidx * kUnitTiles));

        const uint8_t* st = my_stages + sidx * kStageQ4;
        const int pos0 = d.t0 + 16 * kUnitTiles * u;         // position of the unit's first token
        // whether every token counts for every column; if not, ntok[i] tokens of record i do (none of
        // a bad page's)
        const bool full = here == kAll && pos0 + 16 * kUnitTiles <= (kMulti ? min(d.t1, causal_lim + 1) : d.t1);
        int ntok[kUnitTiles];
#pragma unroll
        for (int i = 0; i < kUnitTiles; ++i) ntok[i] = (here >> i) & 1u ? min(16, d.t1 - (pos0 + 16 * i)) : 0;

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

        // ---- online softmax, log2 domain.  lane: tokens gi, gi + 8 x columns 2ti, 2ti + 1 (per n)
        bool grow = false;
        if (!full) {
#pragma unroll
          for (int i = 0; i < kUnitTiles; ++i) {
            const int pos = pos0 + 16 * i + gi;                // this lane's first token; the second is pos + 8
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int last = kMulti ? seen[n][e] : INT_MAX;
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
            top[n][e] *= cs[n][e];
            grow |= top[n][e] > mx[n][e] + (kRescaleThreshold + kPShift);
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
              const float mn = fmaxf(mx[n][e], ceilf(v) - kPShift);      // finite: kNoScore at least
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
              const F2 z = fma2(F2{x[n][i][2 * r], x[n][i][2 * r + 1]}, F2{cs[n][0], cs[n][1]}, F2{-mx[n][0], -mx[n][1]});
              const F2 p = F2{fast_exp2(z.x), fast_exp2(z.y)};
              const F2 sum = add2(F2{l[n][0], l[n][1]}, p);
              l[n][0] = sum.x;
              l[n][1] = sum.y;
              F2 hi = F2{__uint_as_float(__float_as_uint(p.x) & 0xFFFFE000u),
                         __uint_as_float(__float_as_uint(p.y) & 0xFFFFE000u)};
              const F2 lo = add2(p, F2{-hi.x, -hi.y});
              if (kFold) hi = ti < 2 ? hi : lo;
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
      __syncwarp();                // the stage may now be refilled
      sidx ^= 1;
    }

    // ---- merge the warps' states of this item through shared memory, 8 columns at a time.  Each warp
    // writes into its stage that holds no unit in flight (the one it consumed last).
    if (lane == 0) combine_stage[warp] = sidx ^ 1;
    float* my_combine = reinterpret_cast<float*>(my_stages + (sidx ^ 1) * kStageQ4);
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      if (n > 0 && 8 * n >= d.nh) break;                 // uniform: no such columns
      float* cm = my_combine + 8 * kOStride;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[n][e];
#pragma unroll
        for (int dd = 4; dd < 32; dd <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, dd);
        if (gi == 0) {
          cm[2 * ti + e] = mx[n][e];
          cm[8 + 2 * ti + e] = v;
        }
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2*>(my_combine + (2 * ti + e) * kOStride + 16 * gi + 2 * mt) =
              make_float2(o[n][mt][e], o[n][mt][2 + e]);
      }
      consumers_sync<kWarps>();
      for (int hh = warp; hh < 8 && 8 * n + hh < d.nh && !aborted; hh += kWarps) {     // a warp finishes whole columns
        float mw[kWarps];
        float M = kNoScore;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* cwp = reinterpret_cast<const float*>(
              stages + (static_cast<size_t>(w) * kWarpStages + combine_stage[w]) * kStageQ4);
          mw[w] = cwp[8 * kOStride + hh];
          M = fmaxf(M, mw[w]);
        }
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float lsum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* cwp = reinterpret_cast<const float*>(
              stages + (static_cast<size_t>(w) * kWarpStages + combine_stage[w]) * kStageQ4);
          const float f = fast_exp2(mw[w] - M);
          lsum += f * cwp[8 * kOStride + 8 + hh];
          float4 v = *reinterpret_cast<const float4*>(cwp + hh * kOStride + 4 * lane);
          if (kFold) {
            const float4 r = *reinterpret_cast<const float4*>(cwp + (hh + 4) * kOStride + 4 * lane);
            v = make_float4(v.x + r.x, v.y + r.y, v.z + r.z, v.w + r.w);
          }
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
        }
        const size_t bh = static_cast<size_t>(d.b) * a.hq + d.h0 + 8 * n + hh;
        if (d.single) {
          finish_row(a.out, a.lse, query_row(d.b, d.h0 + 8 * n + hh, a.tokens, a.hq), lane, acc, M, lsum, v_factor);
        } else {
          const size_t pidx = bh * a.max_chunks + d.c;
          *reinterpret_cast<float4*>(a.part_o + pidx * ZF_HEAD_DIM + 4 * lane) = acc;
          if (lane == 0) reinterpret_cast<float2*>(a.part_lse)[pidx] = make_float2(M, lsum);
        }
      }
      consumers_sync<kWarps>();
    }
    fence_proxy_async_smem();          // the combine states' stages are refilled by bulk copies
    if (lane == 0) mbar_arrive(&item_empty[buf]);     // this item's metadata and q are free
  }
  // copies still in flight (only after a wait gave up) must land before the CTA exits
  for (int st = 0; st < kWarpStages; ++st)
    if ((inflight >> (st * kUnitTiles)) & kAll) mbar_wait(&my_bars[st], (phase >> st) & 1u);
}

// The merge: one warp per (request, query head, new token).  A partial holds its weighted sum of values as
// it is, its maximum and its sum; the maxima are whole numbers, so the partials' factors are powers of
// two and the merge adds no rounding but those of its sums (a log-sum-exp near 20, kept as one float,
// would be off by 2^-20 in each weight).  Rows with one partial were finished by the attention
// kernel.  The first 32 maxima and kMergePre partial outputs are loaded along with the partial count
// (entries past the count hold anything and are not used).
constexpr int kMergePre = 8;
constexpr int kQ4MergeWarps = 2;
__global__ void __launch_bounds__(kQ4MergeWarps * 32) q4_merge_kernel(const MergeArgs a, const float v_factor) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  allow_next_grid();
  wait_prior_grid();
  const int idx = blockIdx.x * kQ4MergeWarps + warp;
  if (idx >= a.batch * a.hq) return;
  const int b = idx / a.hq, h = idx - b * a.hq;
  const int gq = h / a.group;
  const float2* ml = reinterpret_cast<const float2*>(a.part_lse) + static_cast<size_t>(idx) * a.max_chunks;
  const float4* po = reinterpret_cast<const float4*>(a.part_o + static_cast<size_t>(idx) * a.max_chunks * ZF_HEAD_DIM) + lane;
  const float2 first = lane < a.max_chunks ? ml[lane] : make_float2(kNoScore, 0.f);
  float4 pre[kMergePre];
#pragma unroll
  for (int j = 0; j < kMergePre; ++j)
    pre[j] = j < a.max_chunks ? po[static_cast<size_t>(j) * (ZF_HEAD_DIM / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
  const int nch = a.chunk_counts[(b * (a.hq / a.group) + gq) * a.slices + (h - gq * a.group) / a.hps];
  if (nch == 1) return;
  float M = lane < nch ? first.x : kNoScore;
  for (int i = lane + 32; i < nch; i += 32) M = fmaxf(M, ml[i].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
  const float w0 = lane < nch ? fast_exp2(first.x - M) : 0.f;
  float sum = lane < nch ? w0 * first.y : 0.f;
  for (int i = lane + 32; i < nch; i += 32) sum += fast_exp2(ml[i].x - M) * ml[i].y;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float f, const float4& v) {
    acc.x += f * v.x;
    acc.y += f * v.y;
    acc.z += f * v.z;
    acc.w += f * v.w;
  };
#pragma unroll
  for (int j = 0; j < kMergePre; ++j) {
    const float f = __shfl_sync(0xFFFFFFFFu, w0, j);
    if (j < nch) add(f, pre[j]);
  }
  for (int c0 = 0; c0 < nch; c0 += 32) {
    const float w = c0 == 0 ? w0 : (c0 + lane < nch ? fast_exp2(ml[c0 + lane].x - M) : 0.f);
    const int n = min(32, nch - c0);
    for (int j = c0 == 0 ? kMergePre : 0; j < n; ++j)
      add(__shfl_sync(0xFFFFFFFFu, w, j), po[static_cast<size_t>(c0 + j) * (ZF_HEAD_DIM / 4)]);
  }
  finish_row(a.out, a.lse, query_row(b, h, a.tokens, a.hq), lane, acc, M, sum, v_factor);
}

// 8-column tiles per pass: 1, 2 or 4 (the kernel reads a kv head's records once per 8, 16 or 32 columns).
int q4_col_tiles(int cols) { return cols <= 8 ? 1 : cols <= 16 ? 2 : 4; }

template <int kNT>
Plan q4_plan_nt(int batch, int hq, int hkv, int page_size, int max_pages, int sms) {
  Plan p = make_plan(batch, hq, hkv, page_size, max_pages, sms, Q4Cfg<kNT>::kWarps, 8 * kNT, kItemTilesQ4,
                     kItemTilesQ4);
  const size_t lse = p.part_lse_bytes;               // a partial keeps two floats (maximum and sum) there
  p.part_lse_bytes = (static_cast<size_t>(batch) * hq * p.max_chunks * 8 + 255) & ~static_cast<size_t>(255);
  p.ws_bytes += p.part_lse_bytes - lse;
  return p;
}

Plan q4_plan(int batch, int hq, int hkv, int page_size, int max_pages, int sms) {
  switch (q4_col_tiles(hq / hkv)) {
    case 1: return q4_plan_nt<1>(batch, hq, hkv, page_size, max_pages, sms);
    case 2: return q4_plan_nt<2>(batch, hq, hkv, page_size, max_pages, sms);
    default: return q4_plan_nt<4>(batch, hq, hkv, page_size, max_pages, sms);
  }
}

template <int kNT, bool kMulti, bool kFold = false>
zf_status launch_q4(const AttnArgs& a, float v_factor, int grid, int which, cudaStream_t s) {
  const size_t smem = q4_smem<kNT>(a.batch).total;
  const zf_status st = ensure_smem_limit(reinterpret_cast<const void*>(attn_q4_kernel<kNT, kMulti, kFold>), which, smem);
  if (st != ZF_OK) return st;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Q4Cfg<kNT>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_q4_kernel<kNT, kMulti, kFold>, a, v_factor) == cudaSuccess ? ZF_OK : ZF_ERR_CUDA;
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
  const size_t ws = q4_plan(batch, num_q_heads * tokens, num_kv_heads, page_size, max_pages_per_req, sms).ws_bytes;
  return ws > 0 ? ws : 256;
}

extern "C" zf_status zf_q4_decode_attn(const zf_q4_cache* c, const uint16_t* q, int32_t batch, int32_t tokens,
                                       int32_t num_q_heads, const int32_t* page_table, int32_t max_pages,
                                       const int32_t* seq_lens, float softmax_scale, float* out, float* lse,
                                       void* workspace, size_t workspace_bytes, void* stream) {
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
  // the kernel numbers records with 32 bits
  if (static_cast<unsigned long long>(c->num_pages) * c->num_kv_heads * (c->page_size / 16) >= kNoRecord)
    return ZF_ERR_UNSUPPORTED;
  int sms = 0;
  if ((st = current_sm_count(&sms)) != ZF_OK) return st;
  const int32_t hq = num_q_heads * tokens;
  const int nt = q4_col_tiles(hq / c->num_kv_heads);
  const Plan p = q4_plan(batch, hq, c->num_kv_heads, c->page_size, max_pages, sms);
  if (workspace_bytes < p.ws_bytes) return ZF_ERR_WORKSPACE_TOO_SMALL;

  AttnArgs a{};
  a.k_comp = c->records;
  a.status = c->status;
  a.q = q;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.part_o_bytes);
  a.chunk_counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + p.part_o_bytes + p.part_lse_bytes);
  a.batch = batch;
  a.hq = hq;
  a.hkv = c->num_kv_heads;
  a.group = hq / c->num_kv_heads;
  a.tokens = tokens;
  a.hps = 8 * nt;
  a.slices = p.slices;
  a.page_size = c->page_size;
  a.num_pages = c->num_pages;
  a.max_pages = max_pages;
  a.max_chunks = p.max_chunks;
  a.min_range_pages = p.min_range_pages;
  a.chunk_pages = p.chunk_pages;
  a.scale_log2 = scale_log2;
  a.wait_limit_ns = kWaitTimeoutNs;
  const float v_factor = c->v_scale * kQ4ScaleFactor;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool multi = tokens > 1;
  if (a.group <= 4)
    st = multi ? launch_q4<1, true, true>(a, v_factor, p.grid, 4, s) : launch_q4<1, false, true>(a, v_factor, p.grid, 5, s);
  else if (nt == 1)
    st = multi ? launch_q4<1, true>(a, v_factor, p.grid, 0, s) : launch_q4<1, false>(a, v_factor, p.grid, 1, s);
  else if (nt == 2) st = launch_q4<2, true>(a, v_factor, p.grid, 2, s);
  else st = launch_q4<4, true>(a, v_factor, p.grid, 3, s);
  if (st != ZF_OK) return st;

  MergeArgs m{};
  m.part_o = a.part_o;
  m.part_lse = a.part_lse;
  m.out = out;
  m.lse = lse;
  m.batch = batch;
  m.hq = hq;
  m.chunk_counts = a.chunk_counts;
  m.group = a.group;
  m.slices = a.slices;
  m.max_chunks = p.max_chunks;
  m.tokens = tokens;
  m.hps = a.hps;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  const int rows = batch * hq;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((rows + kQ4MergeWarps - 1) / kQ4MergeWarps);
  cfg.blockDim = dim3(kQ4MergeWarps * 32);
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q4_merge_kernel, m, v_factor) == cudaSuccess ? ZF_OK : ZF_ERR_CUDA;
}
