// zf_verify_drafts: accept drafted tokens against the target's probabilities, and sample one more.
//
// Speculative sampling (Leviathan, Kalman and Matias, "Fast Inference from Transformers via
// Speculative Decoding", 2023): draft x_t stays when u_t q_t(x_t) < p_t(x_t); after the first refusal
// a, one token is drawn from max(p_a - q_a, 0), and from p_n when no draft was refused.  The draw is
// the inverse of the running sum at u_T times the total.
//
// Only the rows that the draw needs are read (one or two per request; the acceptance reads two numbers
// per draft), so the call is bound by 4 or 8 bytes per vocabulary entry and request, and by its chain
// of dependent steps when the batch is small.  A cluster of CTAs (up to 16) owns a request: each
// warp sums a contiguous piece of the row in blocks, the pieces' sums are exchanged through
// distributed shared memory, and the one warp whose piece holds the drawn point finds its block among the
// sums it kept and the entry by reading that block once more, from L2.
//
// Sums are kept as pairs of floats (Knuth's two-sum; 48 bits, 44 and more of them right after the
// additions made here), so the result does not depend on how a row is split, short of a drawn
// point that close to the border between two tokens.  (Double additions would do too, but their rate is
// 1/64 of float's on this GPU: with doubles only above the level of a thread, the call took 41.8 us
// for 64 requests of 128000 entries.)
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <mutex>

#include "zf_device.cuh"
#include "zf_host.h"

namespace zf {

namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 16;
constexpr int kMaxBlocks = 32;                     // blocks of a warp's piece

struct VerifyArgs {
  const float* target;
  const float* draft;
  const int32_t* tokens_in;
  const int32_t* n_drafts;
  const float* uniform;
  const int32_t* token_start;    // kMapped only
  int32_t* accepted;
  int32_t* tokens;
  const int32_t* seq_lens;
  int32_t* out_lens;
  int32_t* status;
  int32_t batch, T, vocab;
};

// Store a sum into the shared memory of CTA `rank` of the cluster, at this CTA's address of `p`.
__device__ __forceinline__ void dsmem_store(float2* p, uint32_t rank, float hi, float lo) {
  uint32_t addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(hi), "f"(lo) : "memory");
}

// What is sampled from: p, or p - q where positive; `drop` names the draft whose q is 1 when there is no q row.
struct Row {
  const float* p;
  const float* q;
  int drop;
};

// An unevaluated sum of two floats, |lo| at most half a step of hi: 48 bits.
struct DF {
  float hi, lo;
};
__device__ __forceinline__ DF two_sum(float a, float b) {          // Knuth: a + b, exactly
  const float s = __fadd_rn(a, b);
  const float z = __fadd_rn(s, -a);
  return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -z)), __fadd_rn(b, -z))};
}
__device__ __forceinline__ DF norm(float s, float e) {             // |s| >= |e|
  const float h = __fadd_rn(s, e);
  return {h, __fadd_rn(e, -__fadd_rn(h, -s))};
}
__device__ __forceinline__ DF add(DF a, DF b) {
  const DF s = two_sum(a.hi, b.hi);
  return norm(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ DF sub(DF a, DF b) { return add(a, {-b.hi, -b.lo}); }
__device__ __forceinline__ bool above(DF a, DF b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ DF shfl(DF v, int lane) {
  return {__shfl_sync(0xFFFFFFFFu, v.hi, lane), __shfl_sync(0xFFFFFFFFu, v.lo, lane)};
}

__device__ __forceinline__ DF warp_sum(DF v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    v = add(v, {__shfl_xor_sync(0xFFFFFFFFu, v.hi, d), __shfl_xor_sync(0xFFFFFFFFu, v.lo, d)});
  return v;
}
// Sums over the lanes up to and including this one.
__device__ __forceinline__ DF warp_scan(DF v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const DF x = {__shfl_up_sync(0xFFFFFFFFu, v.hi, d), __shfl_up_sync(0xFFFFFFFFu, v.lo, d)};
    if (lane >= d) v = add(v, x);
  }
  return v;
}

// A batch: the weights of kBatch consecutive entries from i0 (0 from hi on), kLane per lane, read
// together.  kVec: rows are 16-byte aligned, i0 and hi multiples of 4.  kRuns (and kVec): lane l holds
// entries i0 + 128 k + 4 l .. + 3 as w[4 k ..], else i0 + 32 k + l as w[k].
constexpr int kLane = 16;
constexpr int kBatch = 32 * kLane;
template <bool kVec, bool kHasQ, bool kRuns = kVec>
__device__ __forceinline__ void load_batch(const Row& r, int i0, int hi, int lane, float (&w)[kLane]) {
  float q[kLane];
  if (kVec) {
#pragma unroll
    for (int k = 0; k < kLane / 4; ++k) {
      const int i = i0 + 128 * k + 4 * lane;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (i < hi) {
        x = *reinterpret_cast<const float4*>(r.p + i);
        if (kHasQ) y = *reinterpret_cast<const float4*>(r.q + i);
      }
      w[4 * k] = x.x; w[4 * k + 1] = x.y; w[4 * k + 2] = x.z; w[4 * k + 3] = x.w;
      q[4 * k] = y.x; q[4 * k + 1] = y.y; q[4 * k + 2] = y.z; q[4 * k + 3] = y.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      const int i = kRuns ? i0 + 128 * (k / 4) + 4 * lane + k % 4 : i0 + 32 * k + lane;
      w[k] = i < hi ? r.p[i] : 0.f;
      q[k] = kHasQ && i < hi ? r.q[i] : 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    const int i = kRuns ? i0 + 128 * (k / 4) + 4 * lane + k % 4 : i0 + 32 * k + lane;
    const float x = kHasQ ? w[k] - q[k] : i == r.drop ? w[k] - 1.f : w[k];
    w[k] = x > 0.f ? x : 0.f;
  }
}

// Sum of the weights [lo, hi) by one warp.
template <bool kVec, bool kHasQ>
__device__ __forceinline__ DF block_sum(const Row& r, int lo, int hi, int lane) {
  DF s[2] = {{0.f, 0.f}, {0.f, 0.f}};
  for (int i = lo; i < hi; i += kBatch) {
    float w[kLane];
    load_batch<kVec, kHasQ>(r, i, hi, lane, w);
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      const DF t = two_sum(s[k & 1].hi, w[k]);
      s[k & 1] = {t.hi, __fadd_rn(s[k & 1].lo, t.lo)};
    }
  }
  return warp_sum(add(norm(s[0].hi, s[0].lo), norm(s[1].hi, s[1].lo)));
}

// Sums of a piece's blocks of blen entries into blk; returns their sum.
template <bool kVec, bool kHasQ>
__device__ __forceinline__ DF piece_sum(const Row& r, int lo, int hi, int blen, float2* blk, int lane) {
  DF sum = {0.f, 0.f};
  for (int k = 0, i = lo; i < hi; ++k, i += blen) {
    const DF s = block_sum<kVec, kHasQ>(r, i, min(hi, i + blen), lane);
    if (lane == 0) blk[k] = make_float2(s.hi, s.lo);
    sum = add(sum, s);
  }
  return sum;
}

// The first entry of [lo, hi) with a running sum (from run on) above x; the last positive one when there is
// none.  One warp.
template <bool kVec, bool kHasQ>
__device__ __forceinline__ int scan_block(const Row& r, int lo, int hi, DF run, DF x, int lane) {
  int last = -1;
  for (int i0 = lo; i0 < hi; i0 += kBatch) {
    float w[kLane];
    load_batch<kVec, kHasQ, true>(r, i0, hi, lane, w);
    constexpr int kRun = 4;                            // consecutive entries of a lane: a quarter of the scans
#pragma unroll
    for (int k = 0; k < kLane / kRun; ++k) {
      DF own = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < kRun; ++e) own = add(own, {w[kRun * k + e], 0.f});
      const DF in = warp_scan(own, lane);
      DF at = add(run, sub(in, own));
      int mine = -1, any = -1;                         // this lane's hit, and its last positive entry
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        const float v = w[kRun * k + e];
        at = add(at, {v, 0.f});
        const int i = i0 + 32 * kRun * k + kRun * lane + e;
        if (v > 0.f) {
          any = i;
          if (mine < 0 && above(at, x)) mine = i;
        }
      }
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, mine >= 0), pos = __ballot_sync(0xFFFFFFFFu, any >= 0);
      if (hit) return __shfl_sync(0xFFFFFFFFu, mine, __ffs(hit) - 1);
      if (pos) last = __shfl_sync(0xFFFFFFFFu, any, 31 - __clz(pos));
      run = add(run, shfl(in, 31));
    }
  }
  return last;
}

// Length of each of `parts` equal pieces of n entries, a multiple of 4.
__device__ __forceinline__ int piece_len(int n, int parts) { return ((n + parts - 1) / parts + 3) & ~3; }

// Index of the first of n sums whose running total is above u times the total (the last positive one when
// none is); x: that point, before: the total before the sum found.  -1 when no sum is positive or the
// total is not finite; zero: whether every sum is 0.  One warp, n <= 32 * kPer; given_x: x is given instead.
template <int kPer>
__device__ __forceinline__ int find(const float2* sums, int n, float u, bool given_x, DF& x, DF& before, bool& zero,
                                    int lane) {
  const int per = (n + 31) / 32;
  DF v[kPer], own = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = lane * per + k;
    const float2 s = k < per && i < n ? sums[i] : make_float2(0.f, 0.f);
    v[k] = {s.x, s.y};
    own = add(own, v[k]);
  }
  const DF in = warp_scan(own, lane), total = shfl(in, 31);
  zero = total.hi == 0.f;
  if (!(total.hi > 0.f && total.hi < CUDART_INF_F)) return -1;
  if (!given_x) {
    const float p = __fmul_rn(u, total.hi);
    x = norm(p, __fmaf_rn(u, total.lo, __fmaf_rn(u, total.hi, -p)));
  }
  DF at = sub(in, own), at_mine = at, at_any = at;
  int mine = -1, any = -1;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const DF next = add(at, v[k]);
    if (v[k].hi > 0.f) {
      any = lane * per + k;
      at_any = at;
      if (mine < 0 && above(next, x)) {
        mine = any;
        at_mine = at;
      }
    }
    at = next;
  }
  const uint32_t hit = __ballot_sync(0xFFFFFFFFu, mine >= 0), pos = __ballot_sync(0xFFFFFFFFu, any >= 0);
  const int src = hit ? __ffs(hit) - 1 : 31 - __clz(pos);          // (a positive total has a positive sum)
  before = hit ? shfl(at_mine, src) : shfl(at_any, src);
  return __shfl_sync(0xFFFFFFFFu, hit ? mine : any, src);
}

// Grid: one cluster per request.  kMapped: token_start is given (an instance of its own: 128 x 7 lookups of 50001
// entries without it 13.5 us, 13.9 when the kernel decides while it runs).
template <bool kVec, bool kMapped>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const VerifyArgs a) {
  __shared__ float2 sums[kVerifyMaxCluster * kVerifyWarps];   // of every warp of the cluster
  __shared__ float2 blocks[kVerifyWarps][kMaxBlocks];         // of this CTA's pieces
  __shared__ int sh_piece, sh_zero;
  __shared__ DF sh_x, sh_before;
  __shared__ int sh_acc, sh_n, sh_off;                        // accepted (-1: no places), drafts, places behind the last token's
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int b = blockIdx.x / ranks;
  const int T = a.T, V = a.vocab;
  allow_next_grid();
  wait_prior_grid();
  cluster_sync();           // the cluster's CTAs all run before their shared memory is written

  // ---- accepted drafts (warp 0 of every CTA; T <= 64: two per lane)
  if (warp == 0) {
    // the drafts and their random numbers are read along with the count: two round trips in all
    static_assert(ZF_MAX_TOKENS <= 64, "two drafts per lane");
    int x[2];
    float v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = lane + 32 * k;
      x[k] = t < T ? a.tokens_in[static_cast<size_t>(b) * T + t] : -1;
      v[k] = t < T ? a.uniform[static_cast<size_t>(b) * (T + 1) + t] : 0.f;
    }
    // places that zf_map_tokens gave the request (the last token's, then its drafts'); a count that is no
    // step's is refused like none
    const int places = kMapped ? a.token_start[b + 1] - a.token_start[b] : T + 1;
    const bool idle = kMapped && (places < 1 || places > T + 1);
    const int most = idle ? 0 : places - 1;
    int n = a.n_drafts ? a.n_drafts[b] : most;
    if (idle ? places != 0 : n < 0 || n > most) {
      if (rank == 0 && lane == 0) report(a.status, ZF_DEV_BAD_DRAFT);
    }
    n = min(max(n, 0), most);
    float p[2], q[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = lane + 32 * k;
      const bool in = t < T && x[k] >= 0 && x[k] < V;
      p[k] = in ? a.target[(static_cast<size_t>(b) * (T + 1) + t) * V + x[k]] : 0.f;
      q[k] = in && a.draft ? a.draft[(static_cast<size_t>(b) * T + t) * V + x[k]] : 1.f;
    }
    int acc = n;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = lane + 32 * k;
      const bool bad = x[k] < 0 || x[k] >= V;
      const uint32_t refused = __ballot_sync(0xFFFFFFFFu, t < n && (bad || !(__fmul_rn(v[k], q[k]) < p[k])));
      // (a draft behind the first refused one is not looked at)
      if (acc == n && refused) {
        acc = 32 * k + __ffs(refused) - 1;
        if (rank == 0 && t == acc && bad) report(a.status, ZF_DEV_BAD_DRAFT);
      }
    }
    if (lane == 0) {
      sh_acc = idle ? -1 : acc;
      sh_n = n;
      if (kMapped) sh_off = most;
    }
  }
  __syncthreads();
  const int acc = sh_acc, n = sh_n;
  if (kMapped && acc < 0) {              // the whole cluster: no tokens, and the length stays
    if (rank == 0 && warp == 0) {
      for (int t = lane; t <= T; t += 32) a.tokens[static_cast<size_t>(b) * (T + 1) + t] = -1;
      if (lane == 0) {
        a.accepted[b] = 0;
        if (a.out_lens) a.out_lens[b] = a.seq_lens[b];
      }
    }
    return;
  }
  Row row;
  row.p = a.target + (static_cast<size_t>(b) * (T + 1) + acc) * V;
  row.q = nullptr;
  row.drop = -1;
  if (acc < n) {
    if (a.draft) row.q = a.draft + (static_cast<size_t>(b) * T + acc) * V;
    else row.drop = a.tokens_in[static_cast<size_t>(b) * T + acc];
  }

  // ---- sums of all warps' pieces
  const int len = piece_len(V, ranks * kVerifyWarps);
  const int blen = max((len + kMaxBlocks * kBatch - 1) / (kMaxBlocks * kBatch), 1) * kBatch;
  const int mine = static_cast<int>(rank) * kVerifyWarps + warp;
  const int lo = min(V, mine * len), hi = min(V, lo + len);
  const float u = a.uniform[static_cast<size_t>(b) * (T + 1) + T];
  for (int attempt = 0; attempt < 2; ++attempt) {
    const DF s = row.q ? piece_sum<kVec, true>(row, lo, hi, blen, blocks[warp], lane)
                       : piece_sum<kVec, false>(row, lo, hi, blen, blocks[warp], lane);
    if (lane < static_cast<int>(ranks)) dsmem_store(&sums[mine], lane, s.hi, s.lo);
    cluster_sync();
    if (warp == 0) {                                    // the same in every CTA of the cluster
      DF x, before = {0.f, 0.f};
      bool zero;
      const int piece = find<kVerifyMaxCluster * kVerifyWarps / 32>(sums, ranks * kVerifyWarps, u, false, x, before, zero, lane);
      if (lane == 0) {
        sh_piece = piece;
        sh_zero = zero;
        sh_x = x;
        sh_before = before;
      }
    }
    __syncthreads();
    if (!sh_zero || (!row.q && row.drop < 0)) break;    // uniform over the cluster
    row.q = nullptr;                                    // p nowhere above q: sample from p itself
    row.drop = -1;
    cluster_sync();                                   // the sums have been read everywhere
  }
  const int piece = sh_piece;
  if (piece >= 0 ? piece == mine : mine == 0) {         // one warp of the cluster
    int token = -1;
    if (piece >= 0) {
      // ---- the block of the piece, then the entry in it (read again, from L2)
      DF x = sh_x, inner = {0.f, 0.f};
      DF rest = sub(x, sh_before);
      bool zero;
      const int k = find<kMaxBlocks / 32>(blocks[warp], (hi - lo + blen - 1) / blen, 0.f, true, rest, inner, zero, lane);
      const int blo = lo + max(k, 0) * blen, bhi = min(hi, blo + blen);
      const DF run = add(sh_before, inner);
      token = row.q ? scan_block<kVec, true>(row, blo, bhi, run, x, lane)
                    : scan_block<kVec, false>(row, blo, bhi, run, x, lane);
    } else if (lane == 0) {
      report(a.status, ZF_DEV_BAD_PROBS);
    }
    for (int t = lane; t <= T; t += 32)
      a.tokens[static_cast<size_t>(b) * (T + 1) + t] =
          t < acc ? a.tokens_in[static_cast<size_t>(b) * T + t] : t == acc ? token : -1;
    if (lane == 0) {
      a.accepted[b] = acc;
      if (a.out_lens) {
        const int len = a.seq_lens[b] - ((kMapped ? sh_off : n) - acc);      // (kMapped: places behind its drafts go too)
        if (len < 0) report(a.status, ZF_DEV_BAD_SEQ_LEN);
        a.out_lens[b] = max(len, 0);
      }
    }
  }
  // no CTA reads another's shared memory after the last barrier (the sums were pushed), so none has to wait
}

template <bool kVec, bool kMapped>
zf_status launch_verify(const VerifyArgs& a, int ctas, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * ctas);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;       // (one CTA: a plain launch, 2 us less on the host)
  return cudaLaunchKernelEx(&cfg, verify_kernel<kVec, kMapped>, a) == cudaSuccess ? ZF_OK : ZF_ERR_CUDA;
}

}  // namespace
}  // namespace zf

using namespace zf;

static zf_status verify(int32_t batch, int32_t max_drafts, int32_t vocab, const float* target_probs,
                        const float* draft_probs, const int32_t* draft_tokens, const int32_t* n_drafts,
                        const float* uniform, const int32_t* token_start, int32_t* accepted, int32_t* tokens,
                        const int32_t* seq_lens, int32_t* new_seq_lens, int32_t* status, void* stream) {
  if (batch < 0 || batch > ZF_MAX_BATCH || max_drafts < 1 || max_drafts > ZF_MAX_TOKENS || vocab < 1 ||
      vocab > ZF_MAX_VOCAB)
    return ZF_ERR_INVALID_ARGUMENT;
  if ((seq_lens == nullptr) != (new_seq_lens == nullptr)) return ZF_ERR_INVALID_ARGUMENT;
  if (batch == 0) return ZF_OK;
  if (!target_probs || !draft_tokens || !uniform || !accepted || !tokens) return ZF_ERR_INVALID_ARGUMENT;
  const void* all[] = {target_probs, draft_probs, draft_tokens, n_drafts, uniform, token_start, accepted, tokens,
                       seq_lens, new_seq_lens, status};
  for (const void* p : all)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return ZF_ERR_INVALID_ARGUMENT;
  VerifyArgs a{};
  a.target = target_probs;
  a.draft = draft_probs;
  a.tokens_in = draft_tokens;
  a.n_drafts = n_drafts;
  a.uniform = uniform;
  a.token_start = token_start;
  a.accepted = accepted;
  a.tokens = tokens;
  a.seq_lens = seq_lens;
  a.out_lens = new_seq_lens;
  a.status = status;
  a.batch = batch;
  a.T = max_drafts;
  a.vocab = vocab;
  // CTAs per request: a power of two that brings the grid to 256 CTAs or more (at two per SM most of the GPU's
  // 152), with at least 2048 entries per CTA.
  int ctas = 1;
  while (ctas < kVerifyMaxCluster && batch * ctas < 256 && vocab / (2 * ctas) >= 2048) ctas *= 2;
  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZF_ERR_CUDA;
  if (dev < 0 || dev >= 64) return ZF_ERR_UNSUPPORTED;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      for (const auto kernel : {verify_kernel<true, false>, verify_kernel<false, false>, verify_kernel<true, true>,
                                verify_kernel<false, true>})
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
          return ZF_ERR_CUDA;
      ready[dev] = true;
    }
  }
  const bool vec = vocab % 4 == 0 && aligned16(target_probs) && aligned16(draft_probs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (token_start) return vec ? launch_verify<true, true>(a, ctas, s) : launch_verify<false, true>(a, ctas, s);
  return vec ? launch_verify<true, false>(a, ctas, s) : launch_verify<false, false>(a, ctas, s);
}

extern "C" zf_status zf_verify_drafts(int32_t batch, int32_t max_drafts, int32_t vocab, const float* target_probs,
                                      const float* draft_probs, const int32_t* draft_tokens, const int32_t* n_drafts,
                                      const float* uniform, int32_t* accepted, int32_t* tokens,
                                      const int32_t* seq_lens, int32_t* new_seq_lens, int32_t* status, void* stream) {
  return verify(batch, max_drafts, vocab, target_probs, draft_probs, draft_tokens, n_drafts, uniform, nullptr, accepted,
                tokens, seq_lens, new_seq_lens, status, stream);
}

extern "C" zf_status zf_verify_mapped_drafts(int32_t batch, int32_t max_drafts, int32_t vocab, const float* target_probs,
                                             const float* draft_probs, const int32_t* draft_tokens,
                                             const int32_t* n_drafts, const float* uniform, const int32_t* token_start,
                                             int32_t* accepted, int32_t* tokens, const int32_t* seq_lens,
                                             int32_t* new_seq_lens, int32_t* status, void* stream) {
  if (batch > 0 && !token_start) return ZF_ERR_INVALID_ARGUMENT;
  return verify(batch, max_drafts, vocab, target_probs, draft_probs, draft_tokens, n_drafts, uniform, token_start, accepted,
                tokens, seq_lens, new_seq_lens, status, stream);
}
