// zf_q4_chunk_attn: attention of a ragged batch of new tokens (chunks of prompts, single tokens, or both) over the
// 4-bit paged cache, on the 5th-generation tensor cores.
//
//   x_j = s (q . k_j);  x_j = c tanh(x_j / c) with a cap c;  x_j += slope_h (j - p) with slopes
//   out = sum_j exp(x_j - lse) v_j,  lse = log sum_j exp(x_j)   over  max(0, p - w + 1) <= j <= p
//
// Split.  A unit is a request, a kv head and up to 256 of its query rows (token-major: row r is token r / G, query
// head r % G of the kv head's G), which take the head's records in steps of 128 tokens.  The steps of all units,
// each unit charged kUnitCost more for its start and end, are dealt in equal contiguous ranges to one CTA per SM,
// so ragged batches and long contexts fill the GPU alike; a unit that a border cuts leaves its parts in the
// workspace, which a second kernel joins.
//
// One CTA, 20 warps:
//  * warps 0-3 and 4-7, two softmax groups, a thread per row.  More than 128 rows: group A has rows 0-127, B the
//    rest, and both take every step.  Up to 128 rows: both have the same rows, A the even steps, B the odd ones,
//    and A joins the two at the end from tensor memory (a group's chain from scores to weights is long, so two
//    are under way in either case).  Scores (fp32, 128 x 128) come out of tensor memory twice, for the maximum
//    and for the weights, which go back over them as fp16: the A operand of the second product.  A row's maximum
//    is raised only when a score exceeds it by 2^8 (the output in tensor memory is then rescaled in place).
//  * warps 8-15 decode: warp r takes the 16 tokens of record r of each step from shared memory to the fp16
//    operands.  A code is e2m1 and a scale e4m3, so their product is exact in fp16; K is K-major, V is stored the
//    same way (a token's 8 channels are one row of a core matrix) and read as an MN-major operand.  The operands
//    go round three buffers of 32 KB.
//  * warp 16 issues the products: S = Q K^T (8 x M128 N128 K16 from shared memory) and O += P V (P from tensor
//    memory), alternating between the groups.
//  * warp 17 finds the CTA's range, walks its pieces, resolves pages and starts the records' bulk copies, three
//    steps ahead.
//  * warps 18-19 stage query rows as fp16, each row times a power of two (exact down to 2^-28 of its largest value).
// Every wait is bounded; one that gives up sets ZF_DEV_TIMEOUT and the CTA winds down.
//
// Numbers.  Scores, maxima and sums are fp32.  The weights enter the second product as fp16, 2^7 times their size
// relative to the running maximum (off by at most 2^-11 of themselves down to 2^-21 of it, then by 2^-32 of it): an
// eighth of the error of the result's own rounding to BF16.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <climits>
#include <mutex>

#include "zf_device.cuh"
#include "zf_q4.cuh"

namespace zf {

namespace {

constexpr int kThreads = 640;
constexpr int kDecodeWarp0 = 8, kDecodeWarps = 8;
constexpr int kMmaWarp = 16, kWalkWarp = 17, kQWarp0 = 18, kQWarps = 2;
constexpr int kWarps = kThreads / 32;
constexpr int kStep = 128;                       // tokens per step
constexpr int kUnitRows = 256;                   // query rows per unit
constexpr int kStages = 3;                       // steps of records in flight
constexpr int kRing = 3;                         // operand buffers
constexpr int kOperand = kStep * ZF_HEAD_DIM * 2;
constexpr int kCoreRow = 2048;                   // 8 rows x 128 elements of 16 bits
constexpr int kUnitCost = 2;                     // a unit's start and end in steps
constexpr int kMinCost = 6;                      // a CTA's least share of the steps
constexpr int kSnap = 2;                         // no unit is cut this close to its ends
constexpr float kShift = 7.f;                    // weights are 2^7 times their usual size
constexpr float kBigScore = 1048576.f;           // scores (log2 units) from which differences are taken first
constexpr float kRaise = 8.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2f = 0.6931471805599453f;

// Tensor memory: scores (and weights over them) of A and B, outputs of A and B.
constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemCols = 512;

struct ChunkArgs {
  const uint8_t* records;
  int32_t* status;
  const uint16_t* q;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* token_start;
  const float* slopes;           // [hq] or null
  uint16_t* out;
  float* lse;
  float* part_o;                 // [CTA][2][part_rows][128]
  float2* part_ml;               // [CTA][2][part_rows]: maximum (log2 units) and sum
  int4* part_at;                 // [CTA][2][2]: see write_part
  int32_t batch, rows, hq, hkv, group, page_size, num_pages, max_pages, part_rows, window;
  float scale_log2;              // softmax scale * log2(e) * the decoding's factors
  float cap_log2, inv_cap;       // cap * log2(e), 1 / (cap * log2(e)); kMod only
  float v_factor;
  uint64_t wait_limit_ns;
};

struct Piece {
  int32_t b, g;                  // request (-1: the walk's end), kv head
  int32_t q0;                    // the request's first query row of q (token_start)
  int32_t pos0;                  // position of its first new token
  int32_t row0, rows;            // unit's rows
  int32_t step0, steps;          // steps to take
  int32_t last;                  // tokens the unit's last row sees (tiles at or past it are absent)
  int32_t slot;                  // -1: writes the result; 0, 1: partial slot of the CTA
};

enum : int {
  kBarPieceFull = 0,             // [2]
  kBarPieceEmpty = 2,            // [2]
  kBarRecFull = 4,               // [kStages][8] record landed
  kBarRecEmpty = kBarRecFull + kStages * 8,
  kBarOpFull = kBarRecEmpty + kStages * 8,     // [kRing] operand decoded
  kBarOpEmpty = kBarOpFull + kRing,            // [kRing] its last product done (commit)
  kBarSFull = kBarOpEmpty + kRing,             // [2] scores of a group (commit)
  kBarPFull = kBarSFull + 2,                   // [2] weights of a group
  kBarOFull = kBarPFull + 2,                   // [2] output of a group complete (commit)
  kBarQFull = kBarOFull + 2,
  kBarQEmpty = kBarQFull + 1,                  // last score product of a piece done (commit)
  kBarBDone = kBarQEmpty + 1,                  // group B's part of a shared piece is final
  kBarADone = kBarBDone + 1,                   // group A has read it
  kBarDrain = kBarADone + 1,
  kNumBars = kBarDrain + 1,
};

// Shared memory.  The operand ring comes first: the plan's sums lie over it before the walk begins.
constexpr int kSmRing = 0;
constexpr int kSmQ = kSmRing + kRing * kOperand;
constexpr int kSmRec = kSmQ + 2 * kOperand;
constexpr int kSmScale = kSmRec + kStages * 8 * kQ4Record;     // [2][256] score factors of the rows
constexpr int kSmMl = kSmScale + 2 * kUnitRows * 4;            // [128] float2: group B's maxima and sums
constexpr int kSmPiece = kSmMl + 128 * 8;                      // [2] Piece
constexpr int kSmAbsent = kSmPiece + 2 * 48;                   // [8 steps][8 records] 1: no tokens there
constexpr int kSmBars = kSmAbsent + 64;
constexpr int kSmMisc = kSmBars + kNumBars * 8;                // abort flag, tensor-memory base, range
constexpr int kSmTotal = kSmMisc + 64;
static_assert(kSmTotal <= 227 * 1024 && kSmBars % 8 == 0 && sizeof(Piece) <= 48, "shared memory");
static_assert((ZF_MAX_BATCH + 1) * 8 <= kRing * kOperand, "the plan's sums");

// Instruction descriptor of kind::f16 with FP16 operands and an FP32 accumulator, N 128, M 128; B K-major or
// MN-major (bit 16).
constexpr uint32_t kIdescS = (1u << 4) | (128u / 8 << 17) | (128u / 16 << 24);
constexpr uint32_t kIdescO = kIdescS | (1u << 16);

// Shared-memory descriptors without swizzle of [128][128] operands in core matrices (8 rows x 16 bytes, 128
// contiguous bytes), rows' cores 2048 bytes apart, columns' 128.  K-major (columns along K): leading offset
// 128, stride offset 2048.  MN-major (rows along K): leading offset (along K) 2048, stride offset (along N) 128.
__device__ __forceinline__ uint64_t desc_k(const void* p) { return umma_desc_kmajor(p); }
__device__ __forceinline__ uint64_t desc_mn(const void* p) {
  return static_cast<uint64_t>((smem_addr(p) & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(2048 >> 4) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}

// The MMA warp's issue forms (the whole warp calls, one lane issues).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(kIdescS), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(kIdescO), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
      : "memory");
}

// 32 TMEM lanes (thread t: lane t) x 32 consecutive columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two floats at once (one instruction each).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                              const ChunkArgs& a) {
  if (*abort_flag) return false;
  if (mbar_wait(bar, parity, a.wait_limit_ns)) return true;
  *abort_flag = 1;
  report(a.status, ZF_DEV_TIMEOUT);
  return false;
}

// The same for a whole warp, which takes one outcome.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const ChunkArgs& a) {
  return __all_sync(0xFFFFFFFFu, wait_or_abort(bar, parity, abort_flag, a));
}

// ------------------------------------------------------------------------------------------- plan
struct Request {
  int q0, tokens, len;           // first query row, new tokens, tokens held
};
// Request b, with what lies out of range taken as empty (kReport: and reported).
template <bool kReport>
__device__ __forceinline__ Request request(const ChunkArgs& a, int b) {
  Request r;
  const int s = a.token_start[b], e = a.token_start[b + 1];
  r.q0 = s;
  r.tokens = e - s;
  r.len = a.seq_lens[b];
  bool bad = s < 0 || e < s || e > a.rows;
  if (bad) r.q0 = r.tokens = 0;
  const int most = a.max_pages * a.page_size;
  if (r.len < 0 || r.len > most) {
    bad = true;
    r.len = min(max(r.len, 0), most);
  }
  if (kReport && bad) report(a.status, ZF_DEV_BAD_SEQ_LEN);
  return r;
}
__device__ __forceinline__ int unit_count(const ChunkArgs& a, const Request& r) {
  return (r.tokens * a.group + kUnitRows - 1) / kUnitRows;
}
// Steps [lo, hi) and tokens seen of unit i.
__device__ __forceinline__ void unit_steps(const ChunkArgs& a, const Request& r, int i, int& lo, int& hi, int& last) {
  const int rows = r.tokens * a.group;
  const int t0 = i * kUnitRows / a.group, t1 = (min(rows, (i + 1) * kUnitRows) - 1) / a.group;
  const int p0 = r.len - r.tokens + t0;
  last = max(r.len - r.tokens + t1 + 1, 0);
  hi = (last + kStep - 1) / kStep;
  lo = a.window > 0 ? max(0, p0 + 1 - a.window) / kStep : 0;
  lo = min(lo, hi);
}
__device__ __forceinline__ int unit_cost(const ChunkArgs& a, const Request& r, int i) {
  int lo, hi, last;
  unit_steps(a, r, i, lo, hi, last);
  return hi - lo + kUnitCost;
}

// A place in the order of all steps: unit (b, g, i) and steps of it before the place.
struct Place {
  int b, g, i, s;
};
// The place of cost c (whole warp; sums[b]: cost of the requests before b).
__device__ __forceinline__ Place find_place(const ChunkArgs& a, const long long* sums, long long c, int lane) {
  Place p{a.batch, 0, 0, 0};
  if (c >= sums[a.batch]) return p;
  int lo = 0, hi = a.batch;                          // sums[lo] <= c < sums[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= c) lo = mid; else hi = mid;
  }
  p.b = lo;
  const long long head = (sums[lo + 1] - sums[lo]) / a.hkv;
  long long rest = c - sums[lo];
  p.g = static_cast<int>(rest / head);
  rest -= p.g * head;
  const Request r = request<false>(a, lo);
  const int n = unit_count(a, r);
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane;
    long long in = i < n ? unit_cost(a, r, i) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(0xFFFFFFFFu, in, d);
      if (lane >= d) in += x;
    }
    const uint32_t above = __ballot_sync(0xFFFFFFFFu, i < n && in > rest);
    if (above) {
      const int k = __ffs(above) - 1;
      const long long before = k > 0 ? __shfl_sync(0xFFFFFFFFu, in, k - 1) : 0;
      int slo, shi, last;
      p.i = base + k;
      unit_steps(a, r, p.i, slo, shi, last);
      const int steps = shi - slo;
      int s = static_cast<int>(min(max(rest - before - kUnitCost, 0ll), static_cast<long long>(steps)));
      if (s < kSnap) s = 0;
      else if (steps - s < kSnap) s = steps;
      p.s = s;
      return p;
    }
    rest -= __shfl_sync(0xFFFFFFFFu, in, 31);
  }
  return p;                                          // (not reached: rest < head)
}

// Which rows a partial belongs to: {valid, q0, row0, rows}, {kv head, whether the unit ends here, 0, 0}.
__device__ __forceinline__ void write_part(const ChunkArgs& a, int slot, const Piece* p, bool end) {
  int4* at = a.part_at + (static_cast<size_t>(blockIdx.x) * 2 + slot) * 2;
  at[0] = p ? make_int4(1, p->q0, p->row0, p->rows) : make_int4(0, 0, 0, 0);
  at[1] = p ? make_int4(p->g, end, 0, 0) : make_int4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------------- decode warps
// 16 tokens of K or V from a record to rows 16 r .. of an operand.  Lane (t = lane % 8, q = lane / 8) takes tokens t
// and t + 8, and blocks (16 channels) 2 (t / 2) + {0, 1} + ..: a warp's 8-byte reads of codes then fall on all
// banks, and its 16-byte stores are eight rows of a core matrix each, whatever the block.
template <bool kV>
__device__ __forceinline__ void decode_tile(const uint8_t* rec, uint8_t* op, int r, int lane) {
  const int t = lane & 7, q = lane >> 3;
  uint8_t* base = op + 2 * r * kCoreRow + t * 16;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int block = (2 * (t >> 1) + (q & 1) + 2 * (q >> 1) + 4 * i) & 7;
    const uint32_t sw = *reinterpret_cast<const uint32_t*>(
        rec + (kV ? kQ4VScales + block * 16 + (t >> 1) * 4 : kQ4KScales + t * 16 + (block >> 1) * 4));
    const uint32_t sel = kV ? t & 1 : block & 1;     // byte of token t; that of t + 8 is two on
    const uint32_t two = __byte_perm(sw, 0u, sel | (4u << 4) | ((sel + 2) << 8) | (4u << 12)) << 7;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = t + 8 * h;
      const uint2 codes = *reinterpret_cast<const uint2*>(rec + (kV ? q4_v_code_at(tok, block) : q4_k_code_at(tok, block)));
      const uint32_t one = h ? two >> 16 : two & 0xFFFFu;
      const uint32_t s = (one & 0x3F80u) * 0x10001u;                 // scale byte & 0x7f as a half, twice
      uint32_t x[4], y[4];
      q4_decode4(codes.x, x);
      q4_decode4(codes.y, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = mul_f16x2(x[e], s);
        y[e] = mul_f16x2(y[e], s);
      }
      *reinterpret_cast<uint4*>(base + h * kCoreRow + (2 * block) * 128) = make_uint4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4*>(base + h * kCoreRow + (2 * block + 1) * 128) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}
__device__ __forceinline__ void zero_tile(uint8_t* op, int r, int lane) {
  uint4* at = reinterpret_cast<uint4*>(op + 2 * r * kCoreRow);
#pragma unroll
  for (int i = 0; i < 8; ++i) at[32 * i + lane] = make_uint4(0u, 0u, 0u, 0u);
}

// -------------------------------------------------------------------------------------- softmax
// tanh with an error of a few units in the last place of the larger of it and 2^-12.
__device__ __forceinline__ float tanh_f32(float x) {
  const float ax = fabsf(x);
  const float e = fast_exp2(ax * (2.f * kLog2e));                     // e^{2|x|}
  const float big = 1.f - __fdividef(2.f, e + 1.f);
  const float x2 = x * x;                                             // Taylor series, |x| < 0.35
  const float small =
      fmaf(fmaf(fmaf(fmaf(fmaf(-0.0088632355f, x2, 0.021869488f), x2, -0.053968254f), x2, 0.13333333f), x2, -0.33333333f),
           x2 * ax, ax);
  return copysignf(ax < 0.35f ? small : ax > 15.f ? 1.f : big, x);
}

// A row's scores as they enter the exponential (log2 units): capped, biased, hidden ones -inf.
template <bool kMod>
__device__ __forceinline__ float score(const ChunkArgs& a, float s, float factor, float slope, int far, uint64_t absent, int j,
                                       int window) {
  float x = s * factor;
  if (kMod) {
    if (a.inv_cap > 0.f) x = a.cap_log2 * tanh_f32(x * a.inv_cap);
    x = fmaf(slope, static_cast<float>(-far), x);
  }
  const bool hidden = far < 0 || far >= window || ((absent >> (8 * (j >> 4))) & 1u);
  return hidden ? -CUDART_INF_F : x;
}

template <bool kMod>
__global__ void __launch_bounds__(kThreads, 1) q4_chunk_kernel(const ChunkArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kSmBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kSmMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[kBarPieceFull + i], 1);
      mbar_init(&bars[kBarPieceEmpty + i], kWarps - 1);
      mbar_init(&bars[kBarSFull + i], 1);
      mbar_init(&bars[kBarPFull + i], 4);
      mbar_init(&bars[kBarOFull + i], 1);
    }
    for (int i = 0; i < kStages * 8; ++i) {
      mbar_init(&bars[kBarRecFull + i], 1);
      mbar_init(&bars[kBarRecEmpty + i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bars[kBarOpFull + i], kDecodeWarps);
      mbar_init(&bars[kBarOpEmpty + i], 1);
    }
    mbar_init(&bars[kBarQFull], kQWarps);
    mbar_init(&bars[kBarQEmpty], 1);
    mbar_init(&bars[kBarBDone], 4);
    mbar_init(&bars[kBarADone], 4);
    mbar_init(&bars[kBarDrain], 1);
    *abort_flag = 0;
  }
  fence_mbar_init();
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
  tcgen05_before_sync();
  allow_next_grid();
  wait_prior_grid();

  // ---- costs of the requests (a warp takes 32 at a time; those of many units with all its lanes)
  long long* sums = reinterpret_cast<long long*>(smem + kSmRing);
  for (int base = warp * 32; base < a.batch; base += kThreads) {
    const int b = base + lane;
    Request r{0, 0, 0};
    if (b < a.batch) r = blockIdx.x == 0 ? request<true>(a, b) : request<false>(a, b);
    const int n = unit_count(a, r);
    long long cost = 0;
    if (n <= 4)
      for (int i = 0; i < n; ++i) cost += unit_cost(a, r, i);
    uint32_t many = __ballot_sync(0xFFFFFFFFu, n > 4);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      const Request o{0, __shfl_sync(0xFFFFFFFFu, r.tokens, src), __shfl_sync(0xFFFFFFFFu, r.len, src)};
      const int units = unit_count(a, o);
      long long part = 0;
      for (int i = lane; i < units; i += 32) part += unit_cost(a, o, i);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, d);
      if (lane == src) cost = part;
    }
    if (b < a.batch) sums[b + 1] = cost * a.hkv;
  }
  __syncthreads();
  if (warp == 0) {
    long long carry = 0;
    for (int base = 0; base < a.batch; base += 32) {
      const int b = base + lane;
      long long v = b < a.batch ? sums[b + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += x;
      }
      if (b < a.batch) sums[b + 1] = carry + v;
      carry += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if (lane == 0) sums[0] = 0;
  }
  __syncthreads();
  Place from{a.batch, 0, 0, 0}, to = from;
  if (warp == kWalkWarp) {
    const long long total = sums[a.batch];
    const long long ctas = min(static_cast<long long>(gridDim.x), (total + kMinCost - 1) / kMinCost);
    const long long at = blockIdx.x;
    if (at < ctas) {
      from = find_place(a, sums, total * at / ctas, lane);
      to = find_place(a, sums, total * (at + 1) / ctas, lane);
    }
  }
  tcgen05_after_sync();
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  Piece* pieces = reinterpret_cast<Piece*>(smem + kSmPiece);

  if (warp == kWalkWarp) {
    // ================================================================== walk and copies
    const uint64_t policy = l2_evict_first_policy();
    if (lane == 0) {
      write_part(a, 0, nullptr, false);
      write_part(a, 1, nullptr, false);
    }
    int n = 0;                     // pieces published
    uint32_t gs = 0;               // steps copied
    uint32_t started = 0, phase = 0;       // this lane's copies: stages used, parity of each one's last
    bool ok = true;
    Place at = from;
    bool first = true;
    Request r{0, 0, 0};
    int units = 0;
    bool fresh = true;
    while (ok) {
      // the next request with new tokens
      if (fresh) {
        while (at.b < a.batch) {
          const int b = at.b + lane;
          const Request x = b < a.batch ? request<false>(a, b) : Request{0, 0, 0};
          const uint32_t some = __ballot_sync(0xFFFFFFFFu, x.tokens > 0);
          if (some) {
            const int src = __ffs(some) - 1;
            at.b += src;
            r.q0 = __shfl_sync(0xFFFFFFFFu, x.q0, src);
            r.tokens = __shfl_sync(0xFFFFFFFFu, x.tokens, src);
            r.len = __shfl_sync(0xFFFFFFFFu, x.len, src);
            units = unit_count(a, r);
            break;
          }
          at.b += 32;
        }
        fresh = false;
      }
      const bool final_unit = at.b == to.b && at.g == to.g && at.i == to.i;
      if (at.b >= a.batch || at.b > to.b || (final_unit && to.s == 0)) break;
      Piece p;
      int lo, hi;
      unit_steps(a, r, at.i, lo, hi, p.last);
      const int s0 = first ? at.s : 0, s1 = final_unit ? to.s : hi - lo;
      first = false;
      if (s0 < s1 || hi == lo) {
        p.b = at.b;
        p.g = at.g;
        p.q0 = r.q0;
        p.pos0 = r.len - r.tokens;
        p.row0 = at.i * kUnitRows;
        p.rows = min(r.tokens * a.group - p.row0, kUnitRows);
        p.step0 = lo + s0;
        p.steps = s1 - s0;
        const bool whole = s0 == 0 && s1 == hi - lo;
        p.slot = whole ? -1 : s0 == 0 ? 1 : 0;
        if (!whole && lane == 0) write_part(a, p.slot, &p, s1 == hi - lo);
        const int buf = n & 1;
        ok = n < 2 || wait_warp(&bars[kBarPieceEmpty + buf], ((n >> 1) - 1) & 1, abort_flag, a);
        if (!ok) break;
        if (lane == 0) {
          pieces[buf] = p;
          mbar_arrive(&bars[kBarPieceFull + buf]);
        }
        ++n;
        // its records: lane l resolves the page of tile l of every 4 steps, lanes 0-7 start the copies
        const int32_t* row = a.page_table + static_cast<size_t>(p.b) * a.max_pages;
        auto page_of = [&](int tile) {           // tile: 16 tokens of the context; -1: none there
          if (tile * 16 >= p.last) return -1;
          return row[tile * 16 / a.page_size];
        };
        int next = page_of(p.step0 * 8 + lane);
        for (int s = 0; s < p.steps && ok; s += 4) {
          int cur = next;
          const int tile0 = (p.step0 + s) * 8;
          if ((tile0 + lane) * 16 < p.last && (cur < 0 || cur >= a.num_pages)) {
            report(a.status, ZF_DEV_BAD_PAGE_ID);
            cur = -1;
          }
          next = page_of(tile0 + 32 + lane);
          for (int k = 0; k < 4 && s + k < p.steps; ++k, ++gs) {
            const int page = __shfl_sync(0xFFFFFFFFu, cur, 8 * k + (lane & 7));
            const int stage = gs % kStages;
            const uint32_t use = gs / kStages;
            bool good = true;
            if (lane < 8) {
              good = use == 0 || wait_or_abort(&bars[kBarRecEmpty + stage * 8 + lane], (use - 1) & 1, abort_flag, a);
              if (good) {
                uint64_t* bar = &bars[kBarRecFull + stage * 8 + lane];
                smem[kSmAbsent + (gs & 7) * 8 + lane] = page < 0;
                if (page >= 0) {
                  const int in = ((tile0 + 8 * k + lane) * 16 % a.page_size) >> 4;
                  const uint8_t* src =
                      a.records + ((static_cast<size_t>(page) * a.hkv + p.g) * (a.page_size >> 4) + in) * kQ4Record;
                  mbar_arrive_expect_tx(bar, kQ4Record);
                  bulk_copy_g2s(smem + kSmRec + (stage * 8 + lane) * kQ4Record, src, kQ4Record, bar, policy);
                } else {
                  mbar_arrive(bar);
                }
                started |= 1u << stage;
                phase = (phase & ~(1u << stage)) | ((use & 1) << stage);
              }
            }
            if (!__all_sync(0xFFFFFFFFu, good)) {
              ok = false;
              break;
            }
          }
        }
        if (!ok) break;
      }
      if (final_unit) break;
      if (++at.i >= units) {
        at.i = 0;
        if (++at.g >= a.hkv) {
          at.g = 0;
          ++at.b;
          fresh = true;
        }
      }
    }
    if (ok) {
      const int buf = n & 1;
      ok = n < 2 || wait_warp(&bars[kBarPieceEmpty + buf], ((n >> 1) - 1) & 1, abort_flag, a);
      if (ok && lane == 0) {
        pieces[buf].b = -1;
        mbar_arrive(&bars[kBarPieceFull + buf]);
      }
    }
    // copies in flight must land before the CTA ends (all have, unless a wait gave up)
    for (int k = 0; k < kStages; ++k)
      if ((started >> k & 1) && !mbar_wait(&bars[kBarRecFull + k * 8 + lane], (phase >> k) & 1)) report(a.status, ZF_DEV_TIMEOUT);
    __syncwarp();
  } else if (warp >= kQWarp0) {
    // ================================================================== query rows
    const int w = warp - kQWarp0, t8 = lane & 7, q4 = lane >> 3;
    for (int n = 0;; ++n) {
      const int buf = n & 1;
      if (!wait_warp(&bars[kBarPieceFull + buf], (n >> 1) & 1, abort_flag, a)) break;
      const Piece p = pieces[buf];
      if (p.b < 0) break;
      if (n > 0 && !wait_warp(&bars[kBarQEmpty], (n - 1) & 1, abort_flag, a)) break;
      if (p.steps > 0) {
        float* fac = reinterpret_cast<float*>(smem + kSmScale) + buf * kUnitRows;
        const int groups = (p.rows > 128 ? kUnitRows : 128) / 8;
        const bool negate = a.scale_log2 < 0.f;
#pragma unroll 2
        for (int gr = w; gr < groups; gr += kQWarps) {
          const int rr = gr * 8 + t8;
          uint4 v[4];
          const bool in = rr < p.rows;
          const int row = p.row0 + (in ? rr : 0), tok = row / a.group, h = row - tok * a.group;
          const uint4* src = reinterpret_cast<const uint4*>(
              a.q + (static_cast<size_t>(p.q0 + tok) * a.hq + p.g * a.group + h) * ZF_HEAD_DIM);
          uint32_t big = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = in ? src[q4 + 4 * i] : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t m2 = __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                         __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
            big = max(big, max(m2 & 0xFFFFu, m2 >> 16));
          }
          big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 8));
          big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 16));
          // the power of two that brings the row's largest exponent to 11; the factor takes it back (positive, so
          // that the largest raw score has the largest score: a negative scale negates the row)
          const int k = min(138 - static_cast<int>(big >> 7), 126);
          const float f = __int_as_float(((127 + k) << 23) | (negate ? 0x80000000 : 0));
          if (q4 == 0) fac[rr] = fmaxf(__int_as_float((127 - k) << 23) * fabsf(a.scale_log2), 1e-37f);
          uint8_t* dst = smem + kSmQ + gr * kCoreRow + t8 * 16;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = pack_f16(bf16lo_to_f32(x[e]) * f, bf16hi_to_f32(x[e]) * f);
            *reinterpret_cast<uint4*>(dst + (q4 + 4 * i) * 128) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars[kBarQFull]);
        mbar_arrive(&bars[kBarPieceEmpty + buf]);
      }
      __syncwarp();
    }
  } else if (warp == kMmaWarp) {
    // ================================================================== products
    uint32_t gs = 0;                              // steps before this piece
    uint32_t jobs = 0;                            // parity of the next weights, per group
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int buf = n & 1;
      if (!wait_warp(&bars[kBarPieceFull + buf], (n >> 1) & 1, abort_flag, a)) break;
      const int pb = pieces[buf].b, steps = pieces[buf].steps;
      const bool both = pieces[buf].rows > 128;
      if (pb < 0) break;
      if (!wait_warp(&bars[kBarQFull], n & 1, abort_flag, a)) break;
      tcgen05_after_sync();
      const int N = both ? 2 * steps : steps;
      auto op_wait = [&](uint32_t k) {             // operand k of the ring
        return wait_warp(&bars[kBarOpFull + k % kRing], (k / kRing) & 1, abort_flag, a);
      };
      auto scores = [&](int j) -> bool {
        const int x = j & 1, s = both ? j >> 1 : j;
        const uint32_t k = 2 * (gs + s);
        if (!(both && x) && !op_wait(k)) return false;
        tcgen05_after_sync();
        const uint64_t qa = desc_k(smem + kSmQ + (both && x ? kOperand : 0));
        const uint64_t kb = desc_k(smem + kSmRing + (k % kRing) * kOperand);
#pragma unroll
        for (int e = 0; e < 8; ++e) mma_ss(tmem + kTmemS + 128 * x, qa + e * 16, kb + e * 16, e > 0);
        commit(&bars[kBarSFull + x]);
        if (!both || x) commit(&bars[kBarOpEmpty + k % kRing]);
        if (j == N - 1) commit(&bars[kBarQEmpty]);
        return true;
      };
      auto product = [&](int j) -> bool {
        const int x = j & 1, s = both ? j >> 1 : j;
        const uint32_t k = 2 * (gs + s) + 1;
        if (!(both && x) && !op_wait(k)) return false;
        if (!wait_warp(&bars[kBarPFull + x], (jobs >> x) & 1, abort_flag, a)) return false;
        jobs ^= 1u << x;
        tcgen05_after_sync();
        const uint64_t vb = desc_mn(smem + kSmRing + (k % kRing) * kOperand);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          mma_ts(tmem + kTmemO + 128 * x, tmem + kTmemS + 128 * x + 8 * e, vb + e * (2 * kCoreRow / 16), j > 1 || e > 0);
        if (!both || x) commit(&bars[kBarOpEmpty + k % kRing]);
        if (j >= N - 2) commit(&bars[kBarOFull + x]);
        return true;
      };
      if (N > 0) ok = scores(0);
      if (ok && N > 1) ok = scores(1);
      for (int j = 0; ok && j < N; ++j) {
        ok = product(j);
        if (ok && j + 2 < N) ok = scores(j + 2);
      }
      if (N == 0) commit(&bars[kBarQEmpty]);
      gs += steps;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarPieceEmpty + buf]);
    }
    // every product issued has completed before the tensor memory is given back
    commit(&bars[kBarDrain]);
    if (!mbar_wait(&bars[kBarDrain], 0)) report(a.status, ZF_DEV_TIMEOUT);
  } else if (warp >= kDecodeWarp0) {
    // ================================================================== decoding
    const int r = warp - kDecodeWarp0;
    uint32_t gs = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int buf = n & 1;
      if (!wait_warp(&bars[kBarPieceFull + buf], (n >> 1) & 1, abort_flag, a)) break;
      const int pb = pieces[buf].b, steps = pieces[buf].steps;
      if (pb < 0) break;
      for (int s = 0; s < steps; ++s, ++gs) {
        const int stage = gs % kStages;
        if (!(ok = wait_warp(&bars[kBarRecFull + stage * 8 + r], (gs / kStages) & 1, abort_flag, a))) break;
        const bool absent = *reinterpret_cast<volatile uint8_t*>(smem + kSmAbsent + (gs & 7) * 8 + r) != 0;
        const uint8_t* rec = smem + kSmRec + (stage * 8 + r) * kQ4Record;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t k = 2 * gs + v;
          if (k >= kRing && !(ok = wait_warp(&bars[kBarOpEmpty + k % kRing], (k / kRing - 1) & 1, abort_flag, a))) break;
          uint8_t* op = smem + kSmRing + (k % kRing) * kOperand;
          if (absent) zero_tile(op, r, lane);
          else if (v) decode_tile<true>(rec, op, r, lane);
          else decode_tile<false>(rec, op, r, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarOpFull + k % kRing]);
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(&bars[kBarRecEmpty + stage * 8 + r]);
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&bars[kBarPieceEmpty + buf]);
    }
  } else {
    // ================================================================== softmax
    const int x = warp >> 2;                                  // group
    const int own = 32 * (warp & 3) + lane;                   // row of the 128
    const uint32_t ts = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kTmemS + 128 * x;
    const uint32_t to_x = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kTmemO;
    float2* ml_b = reinterpret_cast<float2*>(smem + kSmMl);
    uint32_t gs = 0, jobs = 0, outs = 0, joins = 0;           // steps before this piece; this group's jobs and outputs; joins
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int buf = n & 1;
      if (!wait_warp(&bars[kBarPieceFull + buf], (n >> 1) & 1, abort_flag, a)) break;
      const Piece p = pieces[buf];
      if (p.b < 0) break;
      const bool both = p.rows > 128;
      const int rr = own + (both ? 128 * x : 0);
      const bool live = rr < p.rows;
      const int row = p.row0 + min(rr, p.rows - 1), tok = row / a.group, h = p.g * a.group + (row - tok * a.group);
      const int pos = p.pos0 + tok;                           // this row's position
      const int window = a.window > 0 ? a.window : INT_MAX;
      // steps of which all rows of the warp see everything: those within these tokens
      const int seen_end = __reduce_min_sync(0xFFFFFFFFu, pos) + 1;
      const int seen_begin = a.window > 0 ? __reduce_max_sync(0xFFFFFFFFu, pos) + 1 - a.window : INT_MIN;
      const float slope = kMod && a.slopes ? a.slopes[h] * kLog2e : 0.f;
      float factor = 0.f, top = -CUDART_INF_F, c = 0.f, sum = 0.f;
      bool any = false;                                       // the output in tensor memory is defined
      const int first = both ? 0 : x, stride = both ? 1 : 2;
      for (int s = first; s < p.steps; s += stride, ++jobs) {
        if (!(ok = wait_warp(&bars[kBarSFull + x], jobs & 1, abort_flag, a))) break;
        tcgen05_after_sync();
        if (s == first) factor = reinterpret_cast<const float*>(smem + kSmScale)[buf * kUnitRows + rr];
        const int t0 = (p.step0 + s) * kStep;
        const uint64_t absent = *reinterpret_cast<volatile uint64_t*>(smem + kSmAbsent + ((gs + s) & 7) * 8);
        bool plain = !kMod && absent == 0 && t0 + kStep <= seen_end && t0 >= seen_begin;
        float mx = -CUDART_INF_F;
        if (plain) {
          float m[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t v[32];
            tmem_ld32(ts + 32 * k, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) m[e & 3] = fmaxf(m[e & 3], __uint_as_float(v[e]));
          }
          mx = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * factor;
          // (scores so large that their rounded differences could pass fp16's range take the other way)
          if (__any_sync(0xFFFFFFFFu, fabsf(mx) >= kBigScore)) plain = false;
        }
        if (!plain) {
          mx = -CUDART_INF_F;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t v[32];
            tmem_ld32(ts + 32 * k, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int j = 32 * k + e;
              const float y = score<kMod>(a, __uint_as_float(v[e]), factor, slope, pos - (t0 + j), absent, j, window);
              mx = fmaxf(mx, y);
              v[e] = __float_as_uint(y);
            }
            tmem_st32(ts + 32 * k, v);
            tmem_wait_st();
          }
        }
        // ---- the maximum
        const bool raise = mx > top + kRaise || (top == -CUDART_INF_F && mx > -CUDART_INF_F);
        if (__any_sync(0xFFFFFFFFu, raise)) {
          float alpha = 1.f;
          if (raise) {
            const float nc = fabsf(mx) < kBigScore ? kShift - mx : -mx;
            alpha = top == -CUDART_INF_F ? 0.f : fast_exp2(nc - c);
            top = mx;
            c = nc;
            sum *= alpha;
          }
          if (any) {
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              uint32_t v[32];
              tmem_ld32(to_x + 128 * x + 32 * k, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
              tmem_st32(to_x + 128 * x + 32 * k, v);
            }
          }
        }
        // ---- weights
        const float mul = plain ? factor : 1.f;
        float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t v[32], w[16];
          tmem_ld32(ts + 32 * k, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 y = fma2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), make_float2(mul, mul),
                            make_float2(c, c));
            y = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            if (e & 1) acc1 = add2(acc1, y); else acc0 = add2(acc0, y);
            w[e] = pack_f16(y.x, y.y);
          }
          tmem_st_32x32b_x16(ts + 16 * k, w);
        }
        acc0 = add2(acc0, acc1);
        sum += acc0.x + acc0.y;
        any = true;
        tmem_wait_st();
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarPFull + x]);
      }
      if (!ok) break;
      // ---- the end of the piece
      const bool has = both ? p.steps > 0 : p.steps > x;
      if (has) {
        if (!wait_warp(&bars[kBarOFull + x], outs++ & 1, abort_flag, a)) break;
        tcgen05_after_sync();
      }
      float fo = 1.f, fb = 0.f;                              // factors of this group's output, and of B's in a shared piece
      bool join = false;
      if (!both && p.steps > 1) {
        if (x == 1) {
          ml_b[own] = make_float2(sum > 0.f || sum != sum ? -c : -CUDART_INF_F, sum);
          tcgen05_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarBDone]);
          if (!wait_warp(&bars[kBarADone], joins++ & 1, abort_flag, a)) break;
        } else {
          if (!wait_warp(&bars[kBarBDone], joins++ & 1, abort_flag, a)) break;
          tcgen05_after_sync();
          join = true;
          const float2 o = ml_b[own];
          const float ma = sum > 0.f || sum != sum ? -c : -CUDART_INF_F;
          const float m = fmaxf(ma, o.x);
          fo = ma == -CUDART_INF_F ? 0.f : fast_exp2(ma - m);
          fb = o.x == -CUDART_INF_F ? 0.f : fast_exp2(o.x - m);
          sum = sum * fo + o.y * fb;
          c = m == -CUDART_INF_F ? 0.f : -m;
        }
      }
      if (both || x == 0) {
        const size_t at = static_cast<size_t>(p.q0 + tok) * a.hq + h;
        const size_t pr = (static_cast<size_t>(blockIdx.x) * 2 + max(p.slot, 0)) * a.part_rows + rr;
        if (p.slot < 0) {
          const float inv = sum == 0.f ? 0.f : a.v_factor / sum;
          fo *= inv;
          fb *= inv;
        }
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          uint32_t v[32];
          if (any) {
            tmem_ld32(to_x + 128 * x + 32 * k, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * fo);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
          if (join) {
            uint32_t u[32];
            tmem_ld32(to_x + 128 + 32 * k, u);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(fmaf(__uint_as_float(u[e]), fb, __uint_as_float(v[e])));
          }
          if (live) {
            if (p.slot < 0) {
              uint4* dst = reinterpret_cast<uint4*>(a.out + at * ZF_HEAD_DIM + 32 * k);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t y[4];
#pragma unroll
                for (int f = 0; f < 4; ++f)
                  y[f] = pack_bf16x2(__uint_as_float(v[8 * e + 2 * f]), __uint_as_float(v[8 * e + 2 * f + 1]));
                dst[e] = make_uint4(y[0], y[1], y[2], y[3]);
              }
            } else {
              uint4* dst = reinterpret_cast<uint4*>(a.part_o + pr * ZF_HEAD_DIM + 32 * k);
#pragma unroll
              for (int e = 0; e < 8; ++e) dst[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
          }
        }
        if (live) {
          const bool none = sum == 0.f;
          if (p.slot < 0) a.lse[at] = none ? -CUDART_INF_F : (log2f(sum) - c) * kLn2f;
          else a.part_ml[pr] = make_float2(none ? -CUDART_INF_F : -c, sum);
        }
        if (join) {
          tcgen05_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarADone]);
        }
      }
      tcgen05_before_sync();
      gs += p.steps;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarPieceEmpty + buf]);
    }
  }

  tcgen05_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tcgen05_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------------------------------- join
// Units that a border between CTAs cut: their first part is in slot 1 of a CTA, the others in slot 0 of the next
// ones, up to the one that ends the unit.  A warp per row, 16 CTAs of 16 rows per possible unit.
constexpr int kJoinRows = 16;
__global__ void __launch_bounds__(512) q4_chunk_join_kernel(const ChunkArgs a, int ctas) {
  allow_next_grid();
  wait_prior_grid();
  const int first = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4* at = a.part_at + (static_cast<size_t>(first) * 2 + 1) * 2;
  const int4 u = at[0];
  const int rr = blockIdx.y * kJoinRows + warp;
  if (!u.x || rr >= u.w) return;
  const int g = at[1].x;
  auto part = [&](int cta, int slot) { return (static_cast<size_t>(cta) * 2 + slot) * a.part_rows + rr; };
  float2 ml = a.part_ml[part(first, 1)];
  float4 o = reinterpret_cast<const float4*>(a.part_o + part(first, 1) * ZF_HEAD_DIM)[lane];
  float m = ml.x, sum = ml.y;
  for (int k = first + 1; k < ctas; ++k) {
    const int4* next = a.part_at + static_cast<size_t>(k) * 4;
    if (!next[0].x) continue;                         // (a CTA whose range was too short to take any step)
    const int end = next[1].y;
    const float2 n = a.part_ml[part(k, 0)];
    const float4 v = reinterpret_cast<const float4*>(a.part_o + part(k, 0) * ZF_HEAD_DIM)[lane];
    const float t = fmaxf(m, n.x);
    if (t > -CUDART_INF_F || t != t) {
      const float f0 = m == -CUDART_INF_F ? 0.f : fast_exp2(m - t), f1 = n.x == -CUDART_INF_F ? 0.f : fast_exp2(n.x - t);
      sum = sum * f0 + n.y * f1;
      o = make_float4(o.x * f0 + v.x * f1, o.y * f0 + v.y * f1, o.z * f0 + v.z * f1, o.w * f0 + v.w * f1);
      m = t;
    }
    if (end) break;
  }
  const int row = u.z + rr, tok = row / a.group, h = g * a.group + (row - tok * a.group);
  const size_t to = static_cast<size_t>(u.y + tok) * a.hq + h;
  const float inv = sum == 0.f ? 0.f : a.v_factor / sum;
  *reinterpret_cast<uint2*>(a.out + to * ZF_HEAD_DIM + 4 * lane) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (lane == 0) a.lse[to] = sum == 0.f ? -CUDART_INF_F : (log2f(sum) + m) * kLn2f;
}

struct ChunkPlan {
  int grid = 1, part_rows = 16;
  size_t o_bytes = 0, ml_bytes = 0, at_bytes = 0;
  size_t bytes() const { return o_bytes + ml_bytes + at_bytes; }
};
ChunkPlan chunk_plan(int rows, int group, int sms) {
  ChunkPlan p;
  p.grid = sms;
  const long long most = static_cast<long long>(rows) * group;
  p.part_rows = static_cast<int>(most < kUnitRows ? (most + 15) / 16 * 16 : kUnitRows);
  const size_t parts = static_cast<size_t>(p.grid) * 2;
  p.o_bytes = parts * p.part_rows * ZF_HEAD_DIM * 4;
  p.ml_bytes = parts * p.part_rows * 8;
  p.at_bytes = parts * 2 * sizeof(int4);
  return p;
}

bool chunk_shape_ok(int batch, int rows, int hq, int hkv, int page_size, int max_pages) {
  if (batch < 0 || batch > ZF_MAX_BATCH || rows < 0 || hkv < 1 || hq < hkv || hq % hkv != 0 || max_pages < 1) return false;
  if (page_size < ZF_BLOCK_TOKENS || page_size % ZF_BLOCK_TOKENS || page_size > ZF_MAX_PAGE_SIZE) return false;
  // positions, and the rows of a request and kv head, are counted with 32 bits
  return static_cast<long long>(max_pages) * page_size < INT_MAX - 16 * kStep &&
         static_cast<long long>(rows) * (hq / hkv) < INT_MAX - 2 * kUnitRows;
}

zf_status sm_count(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZF_ERR_CUDA;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return ZF_ERR_CUDA;
  return ZF_OK;
}

template <typename Kernel, typename... Args>
zf_status launch(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? ZF_OK : ZF_ERR_CUDA;
}

}  // namespace
}  // namespace zf

using namespace zf;

extern "C" size_t zf_q4_chunk_attn_workspace_size(int32_t batch, int32_t rows, int32_t num_q_heads, int32_t num_kv_heads,
                                                  int32_t page_size, int32_t max_pages_per_req) {
  if (!chunk_shape_ok(batch, rows, num_q_heads, num_kv_heads, page_size, max_pages_per_req)) return 0;
  int sms = 0;
  if (sm_count(&sms) != ZF_OK) return 0;
  return chunk_plan(rows, num_q_heads / num_kv_heads, sms).bytes();
}

extern "C" zf_status zf_q4_chunk_attn(const zf_q4_cache* c, const uint16_t* q, int32_t rows, int32_t batch,
                                      int32_t num_q_heads, const int32_t* token_start, const int32_t* page_table,
                                      int32_t max_pages, const int32_t* seq_lens, float softmax_scale, int32_t window,
                                      float softcap, const float* slopes, uint16_t* out, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  zf_status st = check_q4_cache(c);
  if (st != ZF_OK) return st;
  if (!chunk_shape_ok(batch, rows, num_q_heads, c->num_kv_heads, c->page_size, max_pages)) return ZF_ERR_INVALID_ARGUMENT;
  if (window < 0 || !(softcap == 0.f || (softcap >= 1e-3f && softcap <= 1e6f))) return ZF_ERR_INVALID_ARGUMENT;
  if (batch == 0 || rows == 0) return ZF_OK;
  if (!q || !token_start || !page_table || !seq_lens || !out || !lse || !workspace) return ZF_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return ZF_ERR_INVALID_ARGUMENT;
  const void* words[] = {token_start, page_table, seq_lens, slopes, lse};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return ZF_ERR_INVALID_ARGUMENT;
  // the scores' factor, with the cache's scale and the scale decoding's 2^-8 in it, must be a float
  const float scale_log2 = softmax_scale * c->k_scale * (kLog2e * kQ4ScaleFactor);
  if (!(scale_log2 >= -1e37f && scale_log2 <= 1e37f)) return ZF_ERR_INVALID_ARGUMENT;
  int sms = 0;
  if ((st = sm_count(&sms)) != ZF_OK) return st;
  const ChunkPlan p = chunk_plan(rows, num_q_heads / c->num_kv_heads, sms);
  if (workspace_bytes < p.bytes()) return ZF_ERR_WORKSPACE_TOO_SMALL;

  ChunkArgs a{};
  a.records = c->records;
  a.status = c->status;
  a.q = q;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.token_start = token_start;
  a.slopes = slopes;
  a.out = out;
  a.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + p.o_bytes);
  a.part_at = reinterpret_cast<int4*>(ws + p.o_bytes + p.ml_bytes);
  a.batch = batch;
  a.rows = rows;
  a.hq = num_q_heads;
  a.hkv = c->num_kv_heads;
  a.group = num_q_heads / c->num_kv_heads;
  a.page_size = c->page_size;
  a.num_pages = c->num_pages;
  a.max_pages = max_pages;
  a.part_rows = p.part_rows;
  a.window = window;
  a.scale_log2 = scale_log2;
  a.cap_log2 = softcap * kLog2e;
  a.inv_cap = softcap > 0.f ? 1.f / a.cap_log2 : 0.f;
  a.v_factor = c->v_scale * kQ4ScaleFactor;
  a.wait_limit_ns = kWaitTimeoutNs;

  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZF_ERR_CUDA;
  if (dev < 0 || dev >= 64) return ZF_ERR_UNSUPPORTED;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      for (const auto kernel : {q4_chunk_kernel<false>, q4_chunk_kernel<true>})
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmTotal) != cudaSuccess)
          return ZF_ERR_CUDA;
      ready[dev] = true;
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool mod = softcap > 0.f || slopes != nullptr;
  st = mod ? launch(q4_chunk_kernel<true>, dim3(p.grid), kThreads, kSmTotal, s, a)
           : launch(q4_chunk_kernel<false>, dim3(p.grid), kThreads, kSmTotal, s, a);
  if (st != ZF_OK) return st;
  return launch(q4_chunk_join_kernel, dim3(p.grid, p.part_rows / kJoinRows), 512, 0, s, a, p.grid);
}
