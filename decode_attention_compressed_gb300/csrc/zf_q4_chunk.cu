// zf_q4_chunk_attn: attention of a ragged batch of new tokens (chunks of prompts, single tokens, or both) over the
// 4-bit paged cache, on the 5th-generation tensor cores.
//
//   x_j = s (q . k_j);  x_j = c tanh(x_j / c) with a cap c;  x_j += slope_h (j - p) with slopes
//   out = sum_j exp(x_j - lse) v_j,  lse = log sum_j exp(x_j)   over  max(0, p - w + 1) <= j <= p
//
// Split.  A unit is a request, a kv head and up to 256 of its query rows (token-major: row r is token r / G, query
// head r % G of the kv head's G), which take the head's records in steps of 128 tokens.  The steps of all units,
// each unit charged more for its start and end, are dealt in equal contiguous ranges to one CTA per SM,
// so ragged batches and long contexts fill the GPU alike; a unit that a border cuts leaves its parts in the
// workspace, which a second kernel joins.
//
// One CTA, 20 warps:
//  * warps 0-7, softmax: all on the same job, which is a tile of 128 rows and a step, 16 rows a warp, so that a job's
//    chain from scores to weights is short.  Two tiles of up to 256 rows take turns; up to 128 rows, one tile takes
//    one step after the other; up to 16 rows, every warp has them all and one record of the step.  Scores (fp32,
//    128 x 128) come out of tensor memory once; the weights go back over them as fp16, the A operand of the second
//    product.  A row's maximum is raised only when a score exceeds it by 2^8 (the output in tensor memory is then
//    rescaled in place).  These warps also stage query rows as fp16, each row times a power of two (exact down to
//    2^-28 of its largest value).
//  * warps 8-15 decode: warp r takes the 16 tokens of record r of each step from shared memory to the fp16
//    operands.  A code is e2m1 and a scale e4m3, so their product is exact in fp16; K is K-major, V is stored the
//    same way (a token's 8 channels are one row of a core matrix) and read as an MN-major operand.  The operands
//    go round three buffers of 32 KB, or four in units of one tile, where the second query tile's place is free (with
//    three, keys wait for the product two steps before: 64 single tokens 184 us instead of 163).
//  * warp 16 issues the products: S = Q K^T (8 x M128 N128 K16 from shared memory) and O += P V (P from tensor
//    memory).
//  * warp 17 finds the CTA's range, walks its pieces, resolves pages and starts the records' bulk copies, three
//    steps ahead.
// Every wait is bounded; one that gives up sets ZF_DEV_TIMEOUT and the CTA winds down.
//
// Bound.  A product of M128 N128 K16 holds the tensor cores for 64 cycles whatever else runs, so a step's products are
// 2048 cycles with two tiles and 1024 with one; steps take 1.87 and 1.03 us, some 3500 and 2000 cycles.  (One context of
// 131072 tokens and 2048 new ones: 3.09 ms, where its products take 72 % at the measured BF16 rate.)  The rest is the chain
// of a job through the softmax warps (450 cycles until the scores are there, 480 for the maxima, 750 for the weights, with
// 430 of waiting) beside the decoding warps' and the issuing warp's instructions: 0.55 instructions per scheduler and
// cycle.  Without any softmax arithmetic a step would take 8 % less, without decoding as long.  Starting and ending a
// unit costs some 6 us, where instructions that run once wait for themselves, so code is kept short there (query rows
// and output in one place each: mixed batch 447 -> 385 us).
// A cap (up to 128) adds an exponential, a reciprocal and three more operations to each score: a job takes some 3000 cycles
// instead of 1700, the special functions are at 44 % then, so it is the longer chain again (the counters: 0.53 instructions
// per scheduler and cycle, waiting for tensor memory first).
// Measured and not kept: jobs of 64 tokens with two buffers of scores (the issuing warp is the limit: mixed batch 419
// where it was 512, long context 4500 us where it was 3450), two issuing warps, one loop that issues both kinds of units
// (descriptors leave the uniform registers: long context 3270 -> 3560), query rows staged by the decoding warps (385 ->
// 408), spinning waits, skipping warps without rows inside the loop.
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
constexpr int kMmaWarp = 16, kWalkWarp = 17;       // (18 and 19 fill up a warpgroup)
// Registers per thread: the launch's, and what the softmax, decode and other warpgroups (4 warps) make of them (long
// context, prompt: 3094, 469 us with 136 / 64 / 80, 3116, 474 with 144 / 56 / 80, 3090, 469 with 160 / 48 / 64, but then
// 514 instead of 503 with a window and a cap).
constexpr int kRegs = 96, kRegsSoftmax = 136, kRegsDecode = 64, kRegsOther = 80;
static_assert(2 * kRegsSoftmax + 2 * kRegsDecode + kRegsOther <= 5 * kRegs, "a larger sum would wait for registers forever");
constexpr int kStep = 128;                       // tokens per step: of the operands
constexpr int kUnitRows = 256;                   // query rows per unit
constexpr int kFewRows = 16;                     // units of up to so many rows: each warp has them all, and a record of the step
constexpr int kStages = 3;                       // steps of records in flight
constexpr int kRing = 4;                         // operand buffers; the last is the second query tile's in units of two tiles,
                                                 // whose operands go round the first three
constexpr int kOperand = kStep * ZF_HEAD_DIM * 2;
constexpr int kCoreRow = 2048;                   // 8 rows x 128 elements of 16 bits
// What steps, and a unit's start and end, cost with two tiles and with one: a step takes 1.87 us with two tiles and 1.03 with
// one (plain scores, 512 units of 4096 to 16384 tokens); the units' cost was chosen by measurement (mixed batch, prompt: 385,
// 496 us with steps counted alike and two of them per unit; 366, 497 with 14 and 10; 320, 479 with 24 and 18; 312, 475 with 35
// and 20 or 25; 315, 479 with 45 and 30).
constexpr int kStepCost = 7, kStepCost1 = 4, kUnitCost = 35, kUnitCost1 = 20;
constexpr int kMinCost = 29;                     // a CTA's least share (one token over 4000: 20.6 us, with 36 21.8, with 42 22.5)
constexpr int kSnap = 2;                         // no unit is cut this close to its ends
constexpr float kShift = 7.f;                    // weights are 2^7 times their usual size
constexpr float kBigScore = 1048576.f;           // scores (log2 units) from which differences are taken first
constexpr float kRaise = 8.f;
constexpr float kMostCap = 128.f;                // caps up to this: by an exponential (see cap_wide)
constexpr float kLog2e = 1.4426950408889634f, kLn2f = 0.6931471805599453f;

// Tensor memory: two buffers of scores (weights go over them), outputs of the two tiles.
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
  float cap_log2, two_over_cap;  // cap * log2(e), 2 / cap (kCap: scores in log2 units to twice the tanh's argument in them)
  float over_cap;                // 1 / (cap * log2(e)) (kWide: scores in log2 units to the tanh's argument)
  float v_factor;
  uint32_t wait_limit_ns;        // at most 2 s
  int32_t hold;                  // tests: no piece is published before a wait for one has given up
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
  kBarSFull = kBarOpEmpty + kRing,             // [2] scores of a job in a buffer (commit)
  kBarPFull = kBarSFull + 2,                   // [2] its weights
  kBarPvDone = kBarPFull + 2,                  // [2] its product with the values (commit)
  kBarQFull = kBarPvDone + 2,                  // query rows of a piece
  kBarFew = kBarQFull + 1,                     // the softmax warps meet
  kBarDrain = kBarFew + 1,
  kNumBars = kBarDrain + 1,
};

// Shared memory.  The operand ring comes first: the plan's sums lie over it before the walk begins.
constexpr int kSmRing = 0;
constexpr int kSmQ1 = kSmRing + (kRing - 1) * kOperand;
constexpr int kSmQ0 = kSmQ1 + kOperand;
constexpr int kSmRec = kSmQ0 + kOperand;
constexpr int kSmScale = kSmRec + kStages * 8 * kQ4Record;     // [2][256] score factors of the rows
constexpr int kSmPos = kSmScale + 2 * kUnitRows * 4;           // [2][256] their positions
constexpr int kSmSlope = kSmPos + 2 * kUnitRows * 4;           // [2][256] their slopes
constexpr int kSmPlace = kSmSlope + 2 * kUnitRows * 4;         // [2][256] their places among the rows of q and out
constexpr int kSmWhole = kSmPlace + 2 * kUnitRows * 4;         // [2][2][8] int2: steps that all rows of a warp see whole
constexpr int kSmFew = kSmWhole + 2 * 2 * 8 * 8;               // [8 warps][16 rows] float2: c and sum
constexpr int kSmPiece = kSmFew + 8 * kFewRows * 8;             // [2] Piece
constexpr int kSmAbsent = kSmPiece + 2 * 48;                   // [8 steps][8 records] 1: no tokens there
constexpr int kSmBars = kSmAbsent + 64;
constexpr int kSmMisc = kSmBars + kNumBars * 8;                // abort flag, tensor-memory base, range
constexpr int kSmTotal = kSmMisc + 64;
static_assert(kSmTotal <= 227 * 1024 && kSmBars % 8 == 0 && sizeof(Piece) <= 48, "shared memory");
static_assert((ZF_MAX_BATCH + 1) * 4 <= kRing * kOperand, "the plan's sums");

// Instruction descriptors of kind::f16 with FP16 operands and an FP32 accumulator, M 128 and N 128: B K-major, and
// MN-major (bit 16).
constexpr uint32_t kIdescS = (1u << 4) | (128u / 8 << 17) | (128u / 16 << 24);
constexpr uint32_t kIdescO = kIdescS | (1u << 16);

// Shared-memory descriptors without swizzle of [128][128] operands in core matrices (8 rows x 16 bytes, 128
// contiguous bytes), rows' cores 2048 bytes apart, columns' 128.  K-major (columns along K): leading offset
// 128, stride offset 2048.  MN-major (rows along K): leading offset (along K) 2048, stride offset (along N) 128.  The low
// half holds the address and the leading offset (in units of 16 bytes), the high half the stride offset and the version.
constexpr uint32_t kDescHighK = (2048 >> 4) | (1u << 14), kDescHighMn = (128 >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | ((128u >> 4) << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | ((2048u >> 4) << 16); }

template <int kN>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kN));
}
template <int kN>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kN));
}

// The MMA warp's issue forms (the whole warp calls, one lane issues: from a branch of one lane an instruction takes
// about 120 cycles, more than the tensor cores need for it): S = Q K^T over 128 channels, O += P V over 128 tokens.
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e)
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 x, y;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a + 16 * e), "r"(b + 16 * e), "r"(kIdescS), "r"(kDescHighK), "r"(e > 0 ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void mma_weights(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e)
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 y;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 y, {%2, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a + 8 * e), "r"(b + 2 * kCoreRow / 16 * e), "r"(kIdescO), "r"(kDescHighMn), "r"(e > 0 ? 1u : acc)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
      : "memory");
}

// 16 TMEM lanes x 64 columns: thread t gets rows t / 4 and t / 4 + 8, columns 8 j + 2 (t % 4) and + 1 (registers 4 j,
// 4 j + 1 and 4 j + 2, 4 j + 3).
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Stores: 32 columns in the same layout, and 32 columns of pairs of 16 bits (thread t: rows t / 4 and t / 4 + 8, column
// 4 j + t % 4 in registers 2 j and 2 j + 1).
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Loads have arrived; the registers are named, so that nothing that uses them moves ahead of this.
__device__ __forceinline__ void touch(uint32_t (&r)[32]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
               "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
               "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
               "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void touch(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
               "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
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

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// A bounded wait that also ends when another warp's has given up (abort_flag; reported when the CTA ends).  Waits stand in
// some thirty places, so they are short.
__device__ __forceinline__ uint32_t timer_ns() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool wait_longer(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const ChunkArgs& a) {
  const uint32_t t0 = timer_ns();
  while (!*abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    if (timer_ns() - t0 > a.wait_limit_ns) *abort_flag = 1;
  }
  return false;
}
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const ChunkArgs& a) {
  return mbar_try_wait(bar, parity) || wait_longer(bar, parity, abort_flag, a);
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
// Steps [lo, hi) of unit i, and the tokens [first, last) that its rows see.
__device__ __forceinline__ void unit_steps(const ChunkArgs& a, const Request& r, int i, int& lo, int& hi, int& first, int& last) {
  const int rows = r.tokens * a.group;
  const int t0 = i * kUnitRows / a.group, t1 = (min(rows, (i + 1) * kUnitRows) - 1) / a.group;
  const int p0 = r.len - r.tokens + t0;
  last = max(r.len - r.tokens + t1 + 1, 0);
  hi = (last + kStep - 1) / kStep;
  first = a.window > 0 && p0 >= a.window ? p0 + 1 - a.window : 0;       // (p0 may be far below 0)
  lo = min(first / kStep, hi);
}
// Whether unit i has one tile of rows.
__device__ __forceinline__ bool one_tile(const ChunkArgs& a, const Request& r, int i) {
  return r.tokens * a.group - i * kUnitRows <= 128;
}
__device__ __forceinline__ int unit_cost(const ChunkArgs& a, const Request& r, int i) {
  int lo, hi, first, last;
  unit_steps(a, r, i, lo, hi, first, last);
  const int one = one_tile(a, r, i);
  return (hi - lo) * (one ? kStepCost1 : kStepCost) + (one ? kUnitCost1 : kUnitCost);
}

// A place in the order of all steps: unit (b, g, i) and steps of it before the place.
struct Place {
  int b, g, i, s;
};
// The place of cost c (whole warp; sums[b]: cost of the requests before b).
__device__ __forceinline__ Place find_place(const ChunkArgs& a, const int* sums, int c, int lane) {
  Place p{a.batch, 0, 0, 0};
  if (c >= sums[a.batch]) return p;
  int lo = 0, hi = a.batch;                          // sums[lo] <= c < sums[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= c) lo = mid; else hi = mid;
  }
  p.b = lo;
  const int head = (sums[lo + 1] - sums[lo]) / a.hkv;
  int rest = c - sums[lo];
  p.g = rest / head;
  rest -= p.g * head;
  const Request r = request<false>(a, lo);
  const int n = unit_count(a, r);
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane;
    int in = i < n ? unit_cost(a, r, i) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, in, d);
      if (lane >= d) in += x;
    }
    const uint32_t above = __ballot_sync(0xFFFFFFFFu, i < n && in > rest);
    if (above) {
      const int k = __ffs(above) - 1;
      const int before = k > 0 ? __shfl_sync(0xFFFFFFFFu, in, k - 1) : 0;
      int slo, shi, first, last;
      p.i = base + k;
      unit_steps(a, r, p.i, slo, shi, first, last);
      const int steps = shi - slo;
      const bool one = one_tile(a, r, p.i);
      int s = min(max(rest - before - (one ? kUnitCost1 : kUnitCost), 0) / (one ? kStepCost1 : kStepCost), steps);
      if (s < kSnap) s = 0;
      else if (steps - s < kSnap) s = steps;
      p.s = s;
      return p;
    }
    rest -= __shfl_sync(0xFFFFFFFFu, in, 31);
  }
  return p;                                          // (not reached: rest < head)
}

// Lane q of each four has column q of a 4 x 4 matrix and gets row q.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4], int q) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t x = __shfl_xor_sync(0xFFFFFFFFu, q & 1 ? w[i] : w[i + 1], 1);
    if (q & 1) w[i] = x; else w[i + 1] = x;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = __shfl_xor_sync(0xFFFFFFFFu, q & 2 ? w[i] : w[i + 2], 2);
    if (q & 2) w[i] = x; else w[i + 2] = x;
  }
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
  uint32_t sw[2];
  uint2 codes[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {                      // (all loads before the first store, which could be to their place)
    const int block = (2 * (t >> 1) + (q & 1) + 2 * (q >> 1) + 4 * i) & 7;
    sw[i] = *reinterpret_cast<const uint32_t*>(
        rec + (kV ? kQ4VScales + block * 16 + (t >> 1) * 4 : kQ4KScales + t * 16 + (block >> 1) * 4));
#pragma unroll
    for (int h = 0; h < 2; ++h)
      codes[i][h] = *reinterpret_cast<const uint2*>(rec + (kV ? q4_v_code_at(t + 8 * h, block) : q4_k_code_at(t + 8 * h, block)));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int block = (2 * (t >> 1) + (q & 1) + 2 * (q >> 1) + 4 * i) & 7;
    const uint32_t sel = kV ? t & 1 : block & 1;     // byte of token t; that of t + 8 is two on
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t one = __byte_perm(sw[i], 0u, (sel + 2 * h) | 0x4440u);
      const uint32_t s = ((one & 0x7Fu) << 7) * 0x10001u;              // scale byte & 0x7f as a half, twice
      uint32_t x[4], y[4];
      q4_decode4(codes[i][h].x, x);
      q4_decode4(codes[i][h].y, y);
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
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// cap tanh(z) for a pair of z, of any cap: z P(z^2) / Q(z^2) up to |z| = 8.4, where tanh is 1 - 2^-23.  The quotient, a
// minimax fit of tanh(z) / z made for this (least squares, reweighted by the errors), is off by 2^-26.5; its steps round some
// twelve times to 2^-24, so a score is off by at most 2^-20 of itself.  The kernel's other form, cap - 2 cap / (1 + e^(2 z)),
// is off by some 2^-22 of the cap whatever the score: 2^-15 at a cap of 128, which the weights' fp16 hides (2^-11), but 0.09
// at 10^6.  It takes fewer instructions (window and cap: 499 us, with the quotient 599), so it has the caps up to kMostCap.
__device__ __forceinline__ float2 cap_wide(float2 z, float cap) {
  constexpr float kP[] = {0.99999998949508034f, 0.13419579348100072f, 3.541616941987837e-3f, 2.1379765429157377e-5f,
                          1.4457840450921928e-8f};
  constexpr float kQ[] = {1.f, 0.4675290317888972f, 2.6051437834478844e-2f, 3.3614264344577566e-4f, 8.2199561599768221e-7f};
  constexpr float kEnd = 8.4f;
  asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(z.x) : "f"(kEnd));      // (a NaN stays one)
  asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(z.y) : "f"(kEnd));
  const float2 u = mul2(z, z);
  float2 p = make_float2(kP[4], kP[4]), q = make_float2(kQ[4], kQ[4]);
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    p = fma2(p, u, make_float2(kP[i], kP[i]));
    q = fma2(q, u, make_float2(kQ[i], kQ[i]));
  }
  return mul2(mul2(mul2(z, make_float2(cap, cap)), p), make_float2(fast_rcp(q.x), fast_rcp(q.y)));
}

// The columns 8 i + d (i < 16, d < 2) that are at most h, or all; bit 2 i + d.
__device__ __forceinline__ uint32_t bits_to(int h) {
  if (h < 0) return 0u;
  const int n = 2 * (h >> 3) + min((h & 7) + 1, 2);
  return n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}
// Of them those that a row sees, whose position is at column hi: not more than `window` back (0: all), and of records
// (16 columns, a byte each) that are not absent.
__device__ __forceinline__ uint32_t seen_bits(int hi, int window, uint64_t absent) {
  uint32_t m = bits_to(hi);
  if (window > 0) m &= ~bits_to(hi - window);
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if ((absent >> (8 * r)) & 1u) m &= ~(0xFu << (4 * r));
  return m;
}

// What becomes of the scores: nothing, or a cap (kWide: one above kMostCap), slopes, or both.
enum : int { kPlain = 0, kSlope = 1, kCap = 2, kWide = 4 };

// The s-th step that a piece of so many takes.  With slopes the last one first: positive slopes raise the scores with the
// position, so going up a row's maximum would be raised, and its output rescaled, in almost every step (64 single
// tokens: 201 us up, 184 us down).
template <int kMode>
__device__ __forceinline__ int order(int s, int steps) {
  return kMode & kSlope ? steps - 1 - s : s;
}

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1) q4_chunk_kernel(const ChunkArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kSmBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kSmMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[kBarPieceFull + i], 1);
      mbar_init(&bars[kBarPieceEmpty + i], 8 + kDecodeWarps + 1);
      mbar_init(&bars[kBarSFull + i], 1);
      mbar_init(&bars[kBarPFull + i], 8);
      mbar_init(&bars[kBarPvDone + i], 1);
    }
    for (int i = 0; i < kStages * 8; ++i) {
      mbar_init(&bars[kBarRecFull + i], 1);
      mbar_init(&bars[kBarRecEmpty + i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bars[kBarOpFull + i], kDecodeWarps);
      mbar_init(&bars[kBarOpEmpty + i], 1);
    }
    mbar_init(&bars[kBarQFull], 8);
    mbar_init(&bars[kBarFew], 8);
    mbar_init(&bars[kBarDrain], 1);
    *abort_flag = 0;
  }
  fence_mbar_init();
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
  tcgen05_before_sync();
  allow_next_grid();
  wait_prior_grid();

  // ---- costs of the requests (a warp takes 32 at a time; those of many units with all its lanes)
  int* sums = reinterpret_cast<int*>(smem + kSmRing);
  for (int base = warp * 32; base < a.batch; base += kThreads) {
    const int b = base + lane;
    Request r{0, 0, 0};
    if (b < a.batch) r = blockIdx.x == 0 ? request<true>(a, b) : request<false>(a, b);
    const int n = unit_count(a, r);
    int cost = 0;
    if (n <= 4)
      for (int i = 0; i < n; ++i) cost += unit_cost(a, r, i);
    uint32_t many = __ballot_sync(0xFFFFFFFFu, n > 4);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      const Request o{0, __shfl_sync(0xFFFFFFFFu, r.tokens, src), __shfl_sync(0xFFFFFFFFu, r.len, src)};
      const int units = unit_count(a, o);
      int part = 0;
      for (int i = lane; i < units; i += 32) part += unit_cost(a, o, i);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, d);
      if (lane == src) cost = part;
    }
    if (b < a.batch) sums[b + 1] = cost * a.hkv;
  }
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int base = 0; base < a.batch; base += 32) {
      const int b = base + lane;
      int v = b < a.batch ? sums[b + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v, d);
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
    const int total = sums[a.batch];
    const int ctas = min(static_cast<int>(gridDim.x), (total + kMinCost - 1) / kMinCost), at = blockIdx.x;
    if (at < ctas) {
      const int each = total / ctas, more = total - each * ctas;       // the first `more` CTAs take one more
#pragma unroll 1
      for (int k = at; k <= at + 1; ++k) {             // (one place in the code)
        from = to;
        to = find_place(a, sums, each * k + min(k, more), lane);
      }
    }
  }
  tcgen05_after_sync();
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  Piece* pieces = reinterpret_cast<Piece*>(smem + kSmPiece);
  // (a warpgroup's warps run one setmaxnreg together, so it stands before their ways part)
  if (warp >= kMmaWarp) {
  give_registers<kRegsOther>();
  if (warp == kWalkWarp) {
    // ================================================================== walk and copies
    const uint64_t policy = l2_evict_first_policy();
    if (lane == 0) {
      write_part(a, 0, nullptr, false);
      write_part(a, 1, nullptr, false);
    }
    if (a.hold) {
      const uint64_t t0 = global_timer_ns();
      while (!*abort_flag && global_timer_ns() - t0 < 2ull * a.wait_limit_ns + 20000000) __nanosleep(1000);
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
      int lo, hi, from;
      unit_steps(a, r, at.i, lo, hi, from, p.last);
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
          if (tile * 16 >= p.last || tile * 16 + 16 <= from) return -1;
          return row[tile * 16 / a.page_size];
        };
        auto tile_of = [&](int s) {              // lane's tile of the steps from the s-th
          const int o = order<kMode>(s + (lane >> 3), p.steps);
          return o < 0 ? INT_MAX / 16 - 1 : (p.step0 + o) * 8 + (lane & 7);       // (behind every context)
        };
        int next = page_of(tile_of(0));
        // its query rows, for the softmax warps
        for (int i = lane; i < p.rows; i += 32) {
          const int tok = (p.row0 + i) / a.group, h = p.g * a.group + (p.row0 + i - tok * a.group);
          const uint16_t* at_q = a.q + (static_cast<size_t>(p.q0 + tok) * a.hq + h) * ZF_HEAD_DIM;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(at_q));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(at_q + 64));
        }
        for (int s = 0; s < p.steps && ok; s += 4) {
          int cur = next;
          if (tile_of(s) * 16 < p.last && tile_of(s) * 16 + 16 > from && (cur < 0 || cur >= a.num_pages)) {
            report(a.status, ZF_DEV_BAD_PAGE_ID);
            cur = -1;
          }
          next = page_of(tile_of(s + 4));
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
                  const int in = (((p.step0 + order<kMode>(s + k, p.steps)) * 8 + lane) * 16 % a.page_size) >> 4;
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
  } else if (warp == kMmaWarp) {
    // ================================================================== products
    // Job j of a piece: the scores of a tile of 128 rows and a step, and the product of their weights.  More than 128
    // rows: the tiles take turns, each with a buffer of its own; else the one tile's steps alternate between the
    // buffers.  The next job's scores are computed while the softmax has one job's, the one after it once the product
    // that frees their buffer is issued.  Nothing but issuing happens here: waits, commits and instructions cost this
    // warp more cycles than the tensor cores take for a job if they are not few.
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0), sm = __shfl_sync(0xFFFFFFFFu, smem_addr(smem), 0);
    const uint32_t q0 = desc_k(sm + kSmQ0), q1 = desc_k(sm + kSmQ1);
    const uint32_t k0 = desc_k(sm + kSmRing), v0 = desc_mn(sm + kSmRing);
    uint32_t slot = 0, turn = 0;                  // the ring's next operand; parities of the slots' phases
    uint32_t phase = 0;                           // parity of the next weights in each buffer
    uint32_t rows_seen = 0;                       // pieces whose query rows were waited for
    bool ok = true;
    // The next operand's slot (K and V alternate), with the parity of its phase in bit 8.  (The phase before was complete
    // when the operand before it in the slot had been used.)
    auto next = [&](bool both) {
      const uint32_t at = slot | ((turn >> slot) & 1) << 8;
      turn ^= 1u << slot;
      slot = slot + 1 == (both ? kRing - 1 : kRing) ? 0 : slot + 1;
      return at;
    };
    auto decoded = [&](uint32_t at) { return wait_warp(&bars[kBarOpFull + (at & 255)], at >> 8, abort_flag, a); };
    auto weights_ready = [&](int b) {
      const bool good = wait_warp(&bars[kBarPFull + b], (phase >> b) & 1, abort_flag, a);
      phase ^= 1u << b;
      return good;
    };
    for (int n = 0; ok; ++n) {
      const int buf = n & 1;
      if (!wait_warp(&bars[kBarPieceFull + buf], (n >> 1) & 1, abort_flag, a)) break;
      // (the shuffles tell the compiler that these are the same in all lanes: descriptors then stay in uniform registers)
      const int pb = __shfl_sync(0xFFFFFFFFu, pieces[buf].b, 0), steps = __shfl_sync(0xFFFFFFFFu, pieces[buf].steps, 0);
      const bool both = __shfl_sync(0xFFFFFFFFu, pieces[buf].rows, 0) > 128;
      if (pb < 0) break;
      if (steps > 0 && !wait_warp(&bars[kBarQFull], rows_seen++ & 1, abort_flag, a)) break;
      uint32_t k = 0, v = 0;
      if (steps > 0 && both) {
        if (slot == kRing - 1) slot = 0;
        if (!(ok = decoded(k = next(true)))) break;
        k &= 255;
        tcgen05_after_sync();
        mma_scores(tm + kTmemS, q0, k0 + k * (kOperand / 16));
        commit(&bars[kBarSFull]);
        mma_scores(tm + kTmemS + 128, q1, k0 + k * (kOperand / 16));
        commit(&bars[kBarSFull + 1]);
        commit(&bars[kBarOpEmpty + k]);
        for (int s = 0; s < steps; ++s) {
          const bool more = s + 1 < steps;
          if (!(ok = decoded(v = next(true)) && weights_ready(0))) break;
          v &= 255;
          tcgen05_after_sync();
          mma_weights(tm + kTmemO, tm + kTmemS, v0 + v * (kOperand / 16), s > 0);
          if (more) {
            if (!(ok = decoded(k = next(true)))) break;
            k &= 255;
            tcgen05_after_sync();
            mma_scores(tm + kTmemS, q0, k0 + k * (kOperand / 16));
            commit(&bars[kBarSFull]);
          }
          if (!(ok = weights_ready(1))) break;
          tcgen05_after_sync();
          mma_weights(tm + kTmemO + 128, tm + kTmemS + 128, v0 + v * (kOperand / 16), s > 0);
          commit(&bars[kBarOpEmpty + v]);
          if (more) {
            mma_scores(tm + kTmemS + 128, q1, k0 + k * (kOperand / 16));
            commit(&bars[kBarSFull + 1]);
            commit(&bars[kBarOpEmpty + k]);
          }
        }
        if (!ok) break;
        commit(&bars[kBarPvDone]);
        commit(&bars[kBarOpEmpty + kRing - 1]);   // (the second tile's place is free)
      } else if (steps > 0) {
        uint32_t values[2];                       // places of the values of the steps whose scores are under way
        for (int s = 0; s < steps + 2; ++s) {
          const int b = s & 1;
          if (s >= 2) {
            v = b ? values[1] : values[0];
            if (!(ok = decoded(v) && weights_ready(b))) break;
            v &= 255;
            tcgen05_after_sync();
            mma_weights(tm + kTmemO, tm + kTmemS + 128 * b, v0 + v * (kOperand / 16), s > 2);
            commit(&bars[kBarPvDone + b]);
            commit(&bars[kBarOpEmpty + v]);
          }
          if (s < steps) {
            if (!(ok = decoded(k = next(false)))) break;
            k &= 255;
            values[b] = next(false);
            tcgen05_after_sync();
            mma_scores(tm + kTmemS + 128 * b, q0, k0 + k * (kOperand / 16));
            commit(&bars[kBarSFull + b]);
            commit(&bars[kBarOpEmpty + k]);
          }
        }
        if (!ok) break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarPieceEmpty + buf]);
    }
    // every product issued has completed before the tensor memory is given back
    commit(&bars[kBarDrain]);
    if (!mbar_wait(&bars[kBarDrain], 0)) report(a.status, ZF_DEV_TIMEOUT);
  }
  } else if (warp >= kDecodeWarp0) {
    // ================================================================== decoding
    give_registers<kRegsDecode>();
    constexpr int kPerWarp = 8 / kDecodeWarps;       // records of a step
    const int r = warp - kDecodeWarp0;
    uint32_t gs = 0;
    uint32_t slot = 0, turn = 0;                     // the next operand's; parities of the slots' uses
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int buf = n & 1;
      if (!wait_warp(&bars[kBarPieceFull + buf], (n >> 1) & 1, abort_flag, a)) break;
      const int pb = pieces[buf].b, steps = pieces[buf].steps;
      if (pb < 0) break;
      const uint32_t last = pieces[buf].rows > 128 ? kRing - 1 : kRing;
      if (steps > 0 && last < kRing) {
        // the second tile is a use of the last slot (every piece before the last one is done, so no phase is passed over)
        if (slot == last) slot = 0;
        turn ^= 1u << last;
      }
      for (int s = 0; s < steps; ++s, ++gs) {
        const int stage = gs % kStages;
        bool absent[kPerWarp];
#pragma unroll
        for (int i = 0; i < kPerWarp; ++i) {
          const int rec = r + i * kDecodeWarps;
          if (!(ok = wait_warp(&bars[kBarRecFull + stage * 8 + rec], (gs / kStages) & 1, abort_flag, a))) break;
          absent[i] = *reinterpret_cast<volatile uint8_t*>(smem + kSmAbsent + (gs & 7) * 8 + rec) != 0;
        }
        if (!ok) break;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t k = slot;
          // (before the first use: of the phase before the first, which counts as complete)
          if (!(ok = wait_warp(&bars[kBarOpEmpty + k], ((turn >> k) & 1) ^ 1, abort_flag, a))) break;
          turn ^= 1u << k;
          slot = slot + 1 == last ? 0 : slot + 1;
          uint8_t* op = smem + kSmRing + k * kOperand;
#pragma unroll
          for (int i = 0; i < kPerWarp; ++i) {
            const int rec = r + i * kDecodeWarps;
            const uint8_t* at = smem + kSmRec + (stage * 8 + rec) * kQ4Record;
            if (absent[i]) zero_tile(op, rec, lane);
            else if (v) decode_tile<true>(at, op, rec, lane);
            else decode_tile<false>(at, op, rec, lane);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarOpFull + k]);
        }
        if (!ok) break;
        if (lane < kPerWarp) mbar_arrive(&bars[kBarRecEmpty + stage * 8 + r + lane * kDecodeWarps]);
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&bars[kBarPieceEmpty + buf]);
    }
  } else {
    // ================================================================== softmax
    take_registers<kRegsSoftmax>();
    // All eight warps work on the same job, 16 rows of its tile each (warps w and w + 4 share the lanes that they can
    // reach): a lane has rows lane / 4 and lane / 4 + 8 of them, and columns 8 i + 2 (lane % 4), + 1.
    const int row16 = 32 * (warp & 3) + 16 * (warp >> 2);     // the warp's first row in a tile
    const int quad = lane & 3, own = row16 + (lane >> 2);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(row16) << 16);
    float* factors = reinterpret_cast<float*>(smem + kSmScale);
    int* positions = reinterpret_cast<int*>(smem + kSmPos);
    float* slopes = reinterpret_cast<float*>(smem + kSmSlope);
    int* places = reinterpret_cast<int*>(smem + kSmPlace);
    auto whole_of = [&](int buf, int t) -> int2& { return reinterpret_cast<int2*>(smem + kSmWhole)[(buf * 2 + t) * 8 + warp]; };
    uint32_t gs = 0;                                          // steps before this piece
    uint32_t phase = 0, done = 0;                             // parity of the next scores in a buffer; of the products' next end
    // The warp's 16 rows of tile t of the query operand: 4 KB that no other warp writes.
    auto my_q = [&](int t) { return smem + (t ? kSmQ1 : kSmQ0) + (row16 >> 3) * kCoreRow; };

    // Query rows of a piece, 16 of each tile: lane (row lane % 8 of 8, chunks lane / 8 + 4 i of 16 bytes).  (The walk has
    // brought them to L2.)  Up to 16 rows: every warp has the same.
    auto q_rows = [&](int buf) {
      const Piece& p = pieces[buf];
      const int tiles = p.rows > 128 ? 2 : 1, copy = p.rows <= kFewRows ? row16 : 0;
      const bool negate = a.scale_log2 < 0.f, wanted = p.steps > 0;
#pragma unroll 1
      for (int t = 0; t < tiles; ++t) {
        uint4 qv[2][4];
        int low = INT_MAX, high = INT_MIN;
#pragma unroll
        for (int r8 = 0; r8 < 2; ++r8) {
          const int at = 128 * t + row16 + 8 * r8 + (lane & 7);
          const bool in = at - copy < p.rows;
          const int row = p.row0 + min(at - copy, p.rows - 1), tok = row / a.group, h = p.g * a.group + (row - tok * a.group);
          const int place = (p.q0 + tok) * a.hq + h;
          const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<size_t>(place) * ZF_HEAD_DIM);
#pragma unroll
          for (int i = 0; i < 4; ++i) qv[r8][i] = in ? src[(lane >> 3) + 4 * i] : make_uint4(0u, 0u, 0u, 0u);
          low = min(low, p.pos0 + tok);
          high = max(high, p.pos0 + tok);
          if (lane < 8) {
            positions[buf * kUnitRows + at] = p.pos0 + tok;
            places[buf * kUnitRows + at] = place;
            if (kMode & kSlope) slopes[buf * kUnitRows + at] = a.slopes[h] * kLog2e;
          }
        }
        // steps from the first that no row's window cuts to the one that ends at the first row's position or before
        low = __reduce_min_sync(0xFFFFFFFFu, low);
        high = __reduce_max_sync(0xFFFFFFFFu, high);
        const int begin = a.window > 0 && high >= a.window ? (high + 1 - a.window + kStep - 1) / kStep : 0;
        if (lane == 0) whole_of(buf, t) = make_int2(begin, max((low + 1) / kStep - begin, 0));
        if (!wanted) continue;
#pragma unroll
        for (int r8 = 0; r8 < 2; ++r8) {
          uint32_t big = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 x = qv[r8][i];
            const uint32_t m2 = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                         __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
            big = max(big, max(m2 & 0xFFFFu, m2 >> 16));
          }
          big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 8));
          big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 16));
          // the power of two that brings the row's largest exponent to 11; the factor takes it back (positive, so that
          // the largest raw score has the largest score: a negative scale negates the row)
          const int k = min(138 - static_cast<int>(big >> 7), 126);
          const float f = __int_as_float(((127 + k) << 23) | (negate ? 0x80000000 : 0));
          if (lane < 8)
            factors[buf * kUnitRows + 128 * t + row16 + 8 * r8 + lane] =
                fmaxf(__int_as_float((127 - k) << 23) * fabsf(a.scale_log2), 1e-37f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {qv[r8][i].x, qv[r8][i].y, qv[r8][i].z, qv[r8][i].w};
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = pack_f16(bf16lo_to_f32(w[e]) * f, bf16hi_to_f32(w[e]) * f);
            *reinterpret_cast<uint4*>(my_q(t) + r8 * kCoreRow + ((lane >> 3) + 4 * i) * 128 + (lane & 7) * 16) =
                make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      if (!wanted) return;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarQFull]);
    };

    // What a lane keeps of its two rows of a tile.
    struct Rows {
      float c[2], sum[2];                                     // shift - maximum (log2 units), sum of weights
    };
    constexpr float kNone = 1e30f;                            // c before the first score that is seen
    uint32_t met = 0;
    auto meet = [&]() {                                       // all softmax warps
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarFew]);
      return wait_warp(&bars[kBarFew], met++ & 1, abort_flag, a);
    };
    bool ok = true;
    // The end of a piece of up to 16 rows.
    auto finish_few = [&](int buf, Rows& st) {
      // the parts of the output, through the query operand (32 KB, free now) in two halves of 64 channels:
      // [warp][row][64], 8 channels c of row r at c ^ 8 (r & 7)
      float2* rows = reinterpret_cast<float2*>(smem + kSmFew);
      float* parts = reinterpret_cast<float*>(smem + kSmQ0);
      const Piece& p = pieces[buf];
      const int slot = p.slot, live = p.rows;
      const size_t part = (static_cast<size_t>(blockIdx.x) * 2 + max(slot, 0)) * a.part_rows;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        st.sum[r] += __shfl_xor_sync(0xFFFFFFFFu, st.sum[r], 1);
        st.sum[r] += __shfl_xor_sync(0xFFFFFFFFu, st.sum[r], 2);
        if (quad == 0) rows[warp * kFewRows + (lane >> 2) + 8 * r] = make_float2(st.c[r], st.sum[r]);
      }
      if (!(ok = meet())) return;
      float f[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = (lane >> 2) + 8 * r;
        const float2 p0 = rows[2 * quad * kFewRows + row], p1 = rows[(2 * quad + 1) * kFewRows + row];
        float c = fminf(p0.x, p1.x);
        c = fminf(c, __shfl_xor_sync(0xFFFFFFFFu, c, 1));
        c = fminf(c, __shfl_xor_sync(0xFFFFFFFFu, c, 2));
        float sum = p0.y * fast_exp2(c - p0.x) + p1.y * fast_exp2(c - p1.x);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
        const bool none = sum == 0.f;
        f[r] = none ? 0.f : fast_exp2(c - st.c[r]) * (slot >= 0 ? 1.f : a.v_factor / sum);
        if (warp == 0 && quad == 0 && row < live) {
          if (slot < 0) a.lse[places[buf * kUnitRows + row]] = none ? -CUDART_INF_F : (log2f(sum) - c) * kLn2f;
          else a.part_ml[part + row] = make_float2(none ? -CUDART_INF_F : -c, sum);
        }
      }
      const int row = threadIdx.x >> 4, four = threadIdx.x & 15;
#pragma unroll 1
      for (int k = 0; k < 2 && ok; ++k) {
        uint32_t u[32];
        tmem_ld_16x256b_x8(lanes + kTmemO + 64 * k, u);
        tmem_wait_ld();
        touch(u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if ((lane >> 2) + 8 * r < live)
              *reinterpret_cast<float2*>(parts + (warp * kFewRows + (lane >> 2) + 8 * r) * 64 + ((8 * i) ^ (8 * (lane >> 2))) + 2 * quad) =
                  make_float2(__uint_as_float(u[4 * i + 2 * r]) * f[r], __uint_as_float(u[4 * i + 2 * r + 1]) * f[r]);
        if (!(ok = meet())) return;
        if (row < live) {
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(parts + (w * kFewRows + row) * 64 + ((4 * four) ^ (8 * (row & 7))));
            o = make_float4(o.x + x.x, o.y + x.y, o.z + x.z, o.w + x.w);
          }
          if (slot < 0)
            *reinterpret_cast<uint2*>(a.out + static_cast<size_t>(places[buf * kUnitRows + row]) * ZF_HEAD_DIM + 64 * k + 4 * four) =
                make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
          else
            *reinterpret_cast<float4*>(a.part_o + (part + row) * ZF_HEAD_DIM + 64 * k + 4 * four) = o;
        }
        ok = meet();
      }
    };
    // The end of any other piece.
    auto finish = [&](int buf, Rows& st, const Rows& other) {
      const Piece& p = pieces[buf];
      const bool both = p.rows > 128;
      const int steps = p.steps;
#pragma unroll 1
      for (int t = 0; t < (both ? 2 : 1); ++t) {
        const int slot = p.slot, first = 128 * t + row16, live = min(16, p.rows - first);      // rows of this warp
        const size_t part = (static_cast<size_t>(blockIdx.x) * 2 + max(slot, 0)) * a.part_rows;
        float f[2];
        int to[2];                                            // this lane's rows' places in out and lse
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          to[r] = places[buf * kUnitRows + first + (lane >> 2) + 8 * r];
          float sum = st.sum[r];
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
          const bool none = sum == 0.f;
          f[r] = slot >= 0 ? 1.f : none ? 0.f : a.v_factor / sum;
          if (quad == 0 && (lane >> 2) + 8 * r < live) {
            if (slot < 0) a.lse[to[r]] = none ? -CUDART_INF_F : (log2f(sum) - st.c[r]) * kLn2f;
            else a.part_ml[part + first + (lane >> 2) + 8 * r] = make_float2(none ? -CUDART_INF_F : -st.c[r], sum);
          }
        }
        // 64 columns: rows lane / 4 (+ 8), columns 8 i + 2 quad (+ 1)
        auto columns = [&](int k, uint32_t (&u)[32]) {
          if (steps > 0) {
            tmem_ld_16x256b_x8(lanes + kTmemO + 128 * t + 64 * k, u);
            tmem_wait_ld();
            touch(u);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) u[e] = steps > 0 ? __float_as_uint(__uint_as_float(u[e]) * f[(e >> 1) & 1]) : 0u;
        };
        if (slot < 0) {
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            uint32_t u[32];
            columns(k, u);
            // lane q of the four with a row has words q of its 16-byte chunks: it gets chunks q and q + 4
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  w[i] = pack_bf16x2(__uint_as_float(u[4 * (4 * h + i) + 2 * r]), __uint_as_float(u[4 * (4 * h + i) + 2 * r + 1]));
                transpose4(w, quad);
                if ((lane >> 2) + 8 * r < live)
                  reinterpret_cast<uint4*>(a.out + static_cast<size_t>(to[r]) * ZF_HEAD_DIM)[8 * k + 4 * h + quad] =
                      make_uint4(w[0], w[1], w[2], w[3]);
              }
          }
        } else {
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            uint32_t u[32];
            columns(k, u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if ((lane >> 2) + 8 * r < live)
                  *reinterpret_cast<uint2*>(a.part_o + (part + first + (lane >> 2) + 8 * r) * ZF_HEAD_DIM + 64 * k + 8 * i + 2 * quad) =
                      make_uint2(u[4 * i + 2 * r], u[4 * i + 2 * r + 1]);
          }
        }
        st = other;
      }
    };

    // (from -1: the first piece's query rows are read where the next one's are, as instructions that run once wait for
    // themselves longer than for anything else)
    for (int n = -1;; ++n) {
      // (a piece is read from shared memory where it is needed: registers are short in the loop over its jobs)
      const int buf = n & 1;
      const bool both = n >= 0 && pieces[buf].rows > 128;
      const int steps = n >= 0 ? pieces[buf].steps : 0, step0 = pieces[buf].step0, count = both ? 2 * steps : steps;
      Rows st{{kNone, kNone}, {0.f, 0.f}}, other = st;
      const bool few = pieces[buf].rows <= kFewRows && steps > 0;
      if (few) {
        // ---- up to 16 rows.  Every warp has a copy of them and of the tile's 128 rows its 16, and takes the scores of one
        // record, 16 tokens, with a maximum of its own; its weights of the other tokens are 0, so the product leaves
        // its part of the output in its rows, and the parts are summed at the end.  A job's chain from scores to
        // weights, which bounds units of one tile, is half as long (64 single tokens with slopes: 228 -> 201 us).
        const int mine = buf * kUnitRows + own, col0 = 16 * warp + 2 * quad;
        const float factor[2] = {factors[mine], factors[mine + 8]};
        const int pos[2] = {positions[mine], positions[mine + 8]};
        float slope[2] = {0.f, 0.f};
        if (kMode & kSlope) {
          slope[0] = slopes[mine];
          slope[1] = slopes[mine + 8];
        }
        for (int s = 0; s < steps; ++s) {
          const uint32_t b = s & 1, ts = lanes + kTmemS + 128 * b;
          if (!(ok = wait_warp(&bars[kBarSFull + b], (phase >> b) & 1, abort_flag, a))) break;
          phase ^= 1u << b;
          tcgen05_after_sync();
          uint32_t v[8];
          tmem_ld_16x256b_x2(ts + 16 * warp, v);
          const int t0 = (step0 + order<kMode>(s, steps)) * kStep + col0;
          const bool absent = *reinterpret_cast<volatile uint8_t*>(smem + kSmAbsent + ((gs + s) & 7) * 8 + warp) != 0;
          float mul[2] = {kMode == kPlain ? factor[0] : 1.f, kMode == kPlain ? factor[1] : 1.f};
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) asm volatile("" : "+r"(v[e]));
          float mx[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int hi = pos[r] - t0;
            const float base = -slope[r] * static_cast<float>(hi);
            mx[r] = -CUDART_INF_F;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int col = 8 * (e >> 1) + (e & 1);
              uint32_t& at_e = v[4 * (e >> 1) + 2 * r + (e & 1)];
              float x = __uint_as_float(at_e);
              if (kMode & kWide) {
                x *= factor[r] * a.over_cap;
                x = cap_wide(make_float2(x, x), a.cap_log2).x;
              } else if (kMode & kCap) {
                x = fmaf(fast_rcp(1.f + fast_exp2(x * (factor[r] * a.two_over_cap))), -2.f * a.cap_log2, a.cap_log2);
              }
              if (kMode & kSlope) x = fmaf(x, kMode & kCap ? 1.f : factor[r], fmaf(slope[r], static_cast<float>(col), base));
              if (absent || col > hi || (a.window > 0 && col <= hi - a.window)) x = -CUDART_INF_F;
              at_e = __float_as_uint(x);
              mx[r] = fmaxf(mx[r], x);
            }
          }
#pragma unroll
          for (int d = 1; d < 4; d <<= 1) {
            const float x0 = __shfl_xor_sync(0xFFFFFFFFu, mx[0], d), x1 = __shfl_xor_sync(0xFFFFFFFFu, mx[1], d);
            mx[0] = fmaxf(mx[0], x0);
            mx[1] = fmaxf(mx[1], x1);
          }
          bool raise[2];
          float nc[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            mx[r] *= mul[r];
            nc[r] = fabsf(mx[r]) < kBigScore ? kShift - mx[r] : -mx[r];
            raise[r] = nc[r] < st.c[r] - kRaise;
            if (kMode == kPlain && fabsf(mx[r]) >= kBigScore) {       // (multiplied out, see below)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t& at_e = v[4 * (e >> 1) + 2 * r + (e & 1)];
                at_e = __float_as_uint(__uint_as_float(at_e) * mul[r]);
              }
              mul[r] = 1.f;
            }
          }
          if (__any_sync(0xFFFFFFFFu, raise[0] || raise[1])) {
            float alpha[2] = {1.f, 1.f};
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (raise[r]) {
                alpha[r] = fast_exp2(nc[r] - st.c[r]);
                st.c[r] = nc[r];
                st.sum[r] *= alpha[r];
              }
            if (s > 0) {
              if (!(ok = wait_warp(&bars[kBarPvDone + (b ^ 1)], ((done >> (b ^ 1)) & 1) ^ 1, abort_flag, a))) break;
              tcgen05_after_sync();
#pragma unroll 1
              for (int k = 0; k < 4; ++k) {
                uint32_t u[16];
                tmem_ld_16x256b_x4(lanes + kTmemO + 32 * k, u);
                tmem_wait_ld();
                touch(u);
#pragma unroll
                for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha[(e >> 1) & 1]);
                tmem_st_16x256b_x4(lanes + kTmemO + 32 * k, u);
              }
            }
          }
          uint32_t y[4];                                      // [8 i tokens][row]
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = e & 1;
            const float y0 = fast_exp2(fmaf(__uint_as_float(v[2 * e]), mul[r], st.c[r])),
                        y1 = fast_exp2(fmaf(__uint_as_float(v[2 * e + 1]), mul[r], st.c[r]));
            st.sum[r] += y0 + y1;
            y[e] = pack_f16(y0, y1);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = 4 * k + (e >> 2) == warp ? y[e & 3] : 0u;
            tmem_st_16x128b_x8(ts + 32 * k, w);
          }
          tmem_wait_st();
          tcgen05_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarPFull + b]);
          done ^= 1u << b;
        }
      }
      for (int j = few ? count : 0; j < count; ++j) {
        const uint32_t b = j & 1, ts = lanes + kTmemS + 128 * b;
        const int t = both ? j & 1 : 0, s = both ? j >> 1 : j;
        if (!(ok = wait_warp(&bars[kBarSFull + b], (phase >> b) & 1, abort_flag, a))) break;
        phase ^= 1u << b;
        tcgen05_after_sync();
        uint32_t v[2][32];
        tmem_ld_16x256b_x8(ts, v[0]);
        tmem_ld_16x256b_x8(ts + 64, v[1]);
        const int at = buf * kUnitRows + 128 * t + own;
        const float factor[2] = {factors[at], factors[at + 8]};
        const int step = step0 + order<kMode>(s, steps), t0 = step * kStep;
        const int2 range = whole_of(buf, t);
        const bool whole = static_cast<uint32_t>(step - range.x) < static_cast<uint32_t>(range.y) &&
                           *reinterpret_cast<volatile uint64_t*>(smem + kSmAbsent + ((gs + s) & 7) * 8) == 0;
        float mul[2] = {kMode == kPlain ? factor[0] : 1.f, kMode == kPlain ? factor[1] : 1.f};      // scores are mul * v
        tmem_wait_ld();
        touch(v[0]);
        touch(v[1]);
        if (kMode & kWide) {
          const float f[2] = {factor[0] * a.over_cap, factor[1] * a.over_cap};
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float g = f[(e >> 1) & 1];
              const float2 x = cap_wide(mul2(make_float2(__uint_as_float(v[k][e]), __uint_as_float(v[k][e + 1])), make_float2(g, g)), a.cap_log2);
              v[k][e] = __float_as_uint(x.x);
              v[k][e + 1] = __float_as_uint(x.y);
            }
        } else if (kMode & kCap) {
          // cap tanh(s / cap) = cap - 2 cap / (1 + e^(2 s / cap))
          const float f[2] = {factor[0] * a.two_over_cap, factor[1] * a.two_over_cap}, two = -2.f * a.cap_log2;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              v[k][e] = __float_as_uint(fmaf(fast_rcp(1.f + fast_exp2(__uint_as_float(v[k][e]) * f[(e >> 1) & 1])), two, a.cap_log2));
        }
        if (kMode & kSlope) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float slope = slopes[at + 8 * r], base = -slope * static_cast<float>(positions[at + 8 * r] - t0 - 2 * quad);
            const float m = kMode & kCap ? 1.f : factor[r];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
#pragma unroll
                for (int d = 0; d < 2; ++d)
                  v[k][e + 2 * r + d] = __float_as_uint(fmaf(__uint_as_float(v[k][e + 2 * r + d]), m,
                                                             fmaf(slope, static_cast<float>(64 * k + 2 * e + d), base)));
              }
          }
        }
        if (!whole) {
          const uint64_t absent = *reinterpret_cast<volatile uint64_t*>(smem + kSmAbsent + ((gs + s) & 7) * 8);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int hi = positions[at + 8 * r] - t0 - 2 * quad;
            const uint32_t m = seen_bits(hi, a.window, absent);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int n = 0; n < 16; ++n)
                if (!(m & (1u << (16 * k + n)))) v[k][4 * (n >> 1) + 2 * r + (n & 1)] = 0xFF800000u;
          }
        }
        // ---- the rows' maxima, over the four lanes that share them
        float mx[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float m0 = -CUDART_INF_F, m1 = m0;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            m0 = max3(m0, __uint_as_float(v[0][e + 2 * r]), __uint_as_float(v[0][e + 2 * r + 1]));
            m1 = max3(m1, __uint_as_float(v[1][e + 2 * r]), __uint_as_float(v[1][e + 2 * r + 1]));
          }
          mx[r] = fmaxf(m0, m1);
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          const float x0 = __shfl_xor_sync(0xFFFFFFFFu, mx[0], d), x1 = __shfl_xor_sync(0xFFFFFFFFu, mx[1], d);
          mx[0] = fmaxf(mx[0], x0);
          mx[1] = fmaxf(mx[1], x1);
        }
        bool raise[2], big = false;
        float nc[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] *= mul[r];
          nc[r] = fabsf(mx[r]) < kBigScore ? kShift - mx[r] : -mx[r];
          raise[r] = nc[r] < st.c[r] - kRaise;                // (-inf, a row that sees nothing here, raises nothing)
          big |= kMode == kPlain && fabsf(mx[r]) >= kBigScore;
        }
        if (__any_sync(0xFFFFFFFFu, raise[0] || raise[1] || big)) {
          if (kMode == kPlain && __any_sync(0xFFFFFFFFu, big)) {
            // scores so large that their rounded products could pass fp16's range are multiplied out
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 32; ++e) v[k][e] = __float_as_uint(__uint_as_float(v[k][e]) * mul[(e >> 1) & 1]);
            mul[0] = mul[1] = 1.f;
          }
          float alpha[2] = {1.f, 1.f};
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (raise[r]) {
              alpha[r] = fast_exp2(nc[r] - st.c[r]);
              st.c[r] = nc[r];
              st.sum[r] *= alpha[r];
            }
          if (s > 0 && __any_sync(0xFFFFFFFFu, raise[0] || raise[1])) {
            // the output so far in the new units, once the product before this one is in it (with two tiles it was when
            // these scores were complete; with one the product before that was, so its barrier is in this phase or past it)
            if (!both) {
              if (!(ok = wait_warp(&bars[kBarPvDone + (b ^ 1)], ((done >> (b ^ 1)) & 1) ^ 1, abort_flag, a))) break;
              tcgen05_after_sync();
            }
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              uint32_t u[16];
              tmem_ld_16x256b_x4(lanes + kTmemO + 128 * t + 32 * k, u);
              tmem_wait_ld();
              touch(u);
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha[(e >> 1) & 1]);
              tmem_st_16x256b_x4(lanes + kTmemO + 128 * t + 32 * k, u);
            }
          }
        }
        // ---- weights
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int r = e & 1;
            float2 y = fma2(make_float2(__uint_as_float(v[k][2 * e]), __uint_as_float(v[k][2 * e + 1])), make_float2(mul[r], mul[r]),
                            make_float2(st.c[r], st.c[r]));
            y = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            acc[r] = add2(acc[r], y);
            w[e] = pack_f16(y.x, y.y);
          }
          tmem_st_16x128b_x8(ts + 32 * k, w);
        }
        tmem_wait_st();
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarPFull + b]);
        st.sum[0] += acc[0].x + acc[0].y;
        st.sum[1] += acc[1].x + acc[1].y;
        if (both) {
          const Rows x = st;
          st = other;
          other = x;
        } else {
          done ^= 1u << b;
        }
      }
      if (!ok) break;
      // ---- the end of the piece.  The next one's query rows come first, so that its first scores are computed while the
      // output goes out (of up to 16 rows: through the query operand, so before)
      if (!(ok = wait_warp(&bars[kBarPieceFull + (buf ^ 1)], ((n + 1) >> 1) & 1, abort_flag, a))) break;
      const bool more = pieces[buf ^ 1].b >= 0;
      if (steps > 0) {
        // (two tiles: announced once; one: for every step, and the one two before was complete when its scores were)
        if (both) done ^= 1u;
        const uint32_t b = both ? 0 : (count - 1) & 1;
        if (!(ok = wait_warp(&bars[kBarPvDone + b], ((done >> b) & 1) ^ 1, abort_flag, a))) break;
        tcgen05_after_sync();
      }
#pragma unroll 1
      for (int turn = 0; turn < 2 && ok; ++turn) {            // (each once in the code)
        if (turn == static_cast<int>(few)) {
          if (more) q_rows(buf ^ 1);
          continue;
        }
        if (few) {
          finish_few(buf, st);
        } else if (n >= 0) {
          finish(buf, st, other);
        }
      }
      if (!ok) break;
      tcgen05_before_sync();
      gs += steps;
      // ---- the next piece
      __syncwarp();
      if (n >= 0 && lane == 0) mbar_arrive(&bars[kBarPieceEmpty + buf]);
      if (!more) break;
    }
  }

  tcgen05_before_sync();
  __syncthreads();
  if (tid == 0 && *abort_flag) report(a.status, ZF_DEV_TIMEOUT);
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
  // positions and rows (of all heads) are counted with 32 bits
  return static_cast<long long>(max_pages) * page_size < INT_MAX - 16 * kStep &&
         static_cast<long long>(rows) * hq < INT_MAX - 2 * kUnitRows;
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

static zf_status q4_chunk_attn(const zf_q4_cache* c, const uint16_t* q, int32_t rows, int32_t batch, int32_t num_q_heads,
                               const int32_t* token_start, const int32_t* page_table, int32_t max_pages,
                               const int32_t* seq_lens, float softmax_scale, int32_t window, float softcap,
                               const float* slopes, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                               void* stream, uint64_t wait_limit_ns = kWaitTimeoutNs, bool hold = false) {
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
  // the steps of all units, and what a unit is charged besides, are counted with 32 bits
  const long long units = static_cast<long long>(rows) * (num_q_heads / c->num_kv_heads) / kUnitRows + batch;
  if (units * c->num_kv_heads >= INT_MAX ||
      units * c->num_kv_heads * ((static_cast<long long>(max_pages) * c->page_size / kStep + 1) * kStepCost + kUnitCost) >= INT_MAX)
    return ZF_ERR_UNSUPPORTED;
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
  a.two_over_cap = softcap > 0.f ? 2.f / softcap : 0.f;
  a.over_cap = softcap > 0.f ? 1.f / a.cap_log2 : 0.f;
  a.v_factor = c->v_scale * kQ4ScaleFactor;
  a.wait_limit_ns = static_cast<uint32_t>(wait_limit_ns);
  a.hold = hold;

  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZF_ERR_CUDA;
  if (dev < 0 || dev >= 64) return ZF_ERR_UNSUPPORTED;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      for (const auto kernel : {q4_chunk_kernel<kPlain>, q4_chunk_kernel<kSlope>, q4_chunk_kernel<kCap>, q4_chunk_kernel<kCap | kSlope>,
                                q4_chunk_kernel<kCap | kWide>, q4_chunk_kernel<kCap | kWide | kSlope>}) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmTotal) != cudaSuccess)
          return ZF_ERR_CUDA;
        // the warpgroups' shares are those of a launch with kRegs registers per thread
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess) return ZF_ERR_CUDA;
        if (attr.numRegs != kRegs) return ZF_ERR_UNSUPPORTED;
      }
      ready[dev] = true;
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto kernel = softcap > kMostCap ? (slopes ? q4_chunk_kernel<kCap | kWide | kSlope> : q4_chunk_kernel<kCap | kWide>)
                      : softcap > 0.f ? (slopes ? q4_chunk_kernel<kCap | kSlope> : q4_chunk_kernel<kCap>)
                                    : (slopes ? q4_chunk_kernel<kSlope> : q4_chunk_kernel<kPlain>);
  st = launch(kernel, dim3(p.grid), kThreads, kSmTotal, s, a);
  if (st != ZF_OK) return st;
  return launch(q4_chunk_join_kernel, dim3(p.grid, p.part_rows / kJoinRows), 512, 0, s, a, p.grid);
}

extern "C" zf_status zf_q4_chunk_attn(const zf_q4_cache* cache, const uint16_t* q, int32_t rows, int32_t batch,
                                      int32_t num_q_heads, const int32_t* token_start, const int32_t* page_table,
                                      int32_t max_pages, const int32_t* seq_lens, float softmax_scale, int32_t window,
                                      float softcap, const float* slopes, uint16_t* out, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  return q4_chunk_attn(cache, q, rows, batch, num_q_heads, token_start, page_table, max_pages, seq_lens, softmax_scale, window,
                       softcap, slopes, out, lse, workspace, workspace_bytes, stream);
}

extern "C" zf_status zf_q4_chunk_attn_wait_test(const zf_q4_cache* cache, const uint16_t* q, int32_t rows, int32_t batch,
                                                int32_t num_q_heads, const int32_t* token_start,
                                                const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                                                float softmax_scale, int32_t window, float softcap, const float* slopes,
                                                uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                                uint64_t wait_limit_ns, void* stream) {
  if (wait_limit_ns < 1000 || wait_limit_ns > kWaitTimeoutNs) return ZF_ERR_INVALID_ARGUMENT;
  return q4_chunk_attn(cache, q, rows, batch, num_q_heads, token_start, page_table, max_pages, seq_lens, softmax_scale, window,
                       softcap, slopes, out, lse, workspace, workspace_bytes, stream, wait_limit_ns, true);
}
