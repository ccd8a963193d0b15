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
// warp sums a contiguous piece of the row, the sums of all warps are exchanged through distributed
// shared memory, and the one CTA whose piece holds the drawn point narrows it down (its
// warps re-read that warp's piece from L2, then one warp the piece of a piece).
//
// Sums: a thread adds its weights in float with the rounding errors carried along (Knuth's two-sum,
// 48 bits), everything above that is double.  The result so does not depend on how the row is split,
// short of a drawn point that falls within 2^-44 of the border between two tokens.  (Double
// additions for every weight would bind the call: their rate is 1/64 of float's here.)
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "zf_device.cuh"
#include "zf_host.h"

namespace zf {

namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 16;

struct VerifyArgs {
  const float* target;
  const float* draft;
  const int32_t* tokens_in;
  const int32_t* n_drafts;
  const float* uniform;
  int32_t* accepted;
  int32_t* tokens;
  const int32_t* seq_lens;
  int32_t* out_lens;
  int32_t* status;
  int32_t batch, T, vocab;
};

__device__ __forceinline__ void v_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Store a double into the shared memory of CTA `rank` of the cluster, at this CTA's address of `p`.
__device__ __forceinline__ void dsmem_store(double* p, uint32_t rank, double v) {
  uint32_t addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// What is sampled from: p, or p - q where positive; `drop` names the draft whose q is 1 when there is no q row.
struct Row {
  const float* p;
  const float* q;
  int drop;
};

__device__ __forceinline__ float weight(const Row& r, int i, float p, float q) {
  float w = r.q ? p - q : (i == r.drop ? p - 1.f : p);
  return w > 0.f ? w : 0.f;
}
__device__ __forceinline__ float weight_at(const Row& r, int i) { return weight(r, i, r.p[i], r.q ? r.q[i] : 0.f); }

struct Sum {
  float s = 0.f, e = 0.f;
  __device__ __forceinline__ void add(float w) {          // s + e gains w, the rounding error of s in e
    const float t = __fadd_rn(s, w);
    const float z = __fadd_rn(t, -s);
    e = __fadd_rn(e, __fadd_rn(__fadd_rn(s, -__fadd_rn(t, -z)), __fadd_rn(w, -z)));
    s = t;
  }
  __device__ __forceinline__ double value() const { return static_cast<double>(s) + static_cast<double>(e); }
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// Sum of the weights [lo, hi) by one warp.  kVec: rows are 16-byte aligned, lo and hi multiples of 4.
template <bool kVec>
__device__ __forceinline__ double piece_sum(const Row& r, int lo, int hi, int lane) {
  Sum s;
  if (kVec) {
#pragma unroll 4
    for (int i = lo + 4 * lane; i < hi; i += 128) {
      const float4 p = *reinterpret_cast<const float4*>(r.p + i);
      const float4 q = r.q ? *reinterpret_cast<const float4*>(r.q + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      s.add(weight(r, i, p.x, q.x));
      s.add(weight(r, i + 1, p.y, q.y));
      s.add(weight(r, i + 2, p.z, q.z));
      s.add(weight(r, i + 3, p.w, q.w));
    }
  } else {
#pragma unroll 8
    for (int i = lo + lane; i < hi; i += 32) s.add(weight_at(r, i));
  }
  return warp_sum(s.value());
}

// Length of each of `parts` equal pieces of n entries, a multiple of 4.
__device__ __forceinline__ int piece_len(int n, int parts) { return ((n + parts - 1) / parts + 3) & ~3; }

// Index of the first of n sums whose running total is above r (the last positive one when none is), and
// the total before it; -1 when no sum is positive.  One warp; n <= 32 * kVerifyMaxCluster.
__device__ __forceinline__ int find(const double* sums, int n, double r, double& before, int lane) {
  double run = 0.0, last_before = 0.0;
  int last = -1;
  for (int b = 0; b < n; b += 32) {
    const double v = b + lane < n ? sums[b + lane] : 0.0;
    double in = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double x = __shfl_up_sync(0xFFFFFFFFu, in, d);
      if (lane >= d) in += x;
    }
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, v > 0.0 && run + in > r);
    const uint32_t pos = __ballot_sync(0xFFFFFFFFu, v > 0.0);
    const uint32_t pick = hit ? hit & (0u - hit) : pos;      // the first hit, or the last positive
    if (pick) {
      const int at = 31 - __clz(pick);
      last = b + at;
      last_before = run + __shfl_sync(0xFFFFFFFFu, in - v, at);
      if (hit) break;
    }
    run += __shfl_sync(0xFFFFFFFFu, in, 31);
  }
  before = last_before;
  return last;
}

// Grid: one cluster per request.
template <bool kVec>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyArgs a) {
  __shared__ double sums[kVerifyMaxCluster * kVerifyWarps];   // of every warp of the cluster
  __shared__ double part[kVerifyWarps];
  __shared__ int sh_acc, sh_n;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int b = blockIdx.x / ranks;
  const int T = a.T, V = a.vocab;
  allow_next_grid();
  wait_prior_grid();
  v_cluster_sync();           // the cluster's CTAs all run before their shared memory is written

  // ---- accepted drafts (warp 0 of every CTA; T <= 64: two per lane)
  if (warp == 0) {
    int n = a.n_drafts ? a.n_drafts[b] : T;
    if (n < 0 || n > T) {
      if (rank == 0 && lane == 0) report(a.status, ZF_DEV_BAD_DRAFT);
      n = min(max(n, 0), T);
    }
    int acc = n;
    for (int t0 = 0; t0 < n; t0 += 32) {
      const int t = t0 + lane;
      bool ok = true;
      if (t < n) {
        const int x = a.tokens_in[static_cast<size_t>(b) * T + t];
        if (x < 0 || x >= V) {
          ok = false;
          if (rank == 0) report(a.status, ZF_DEV_BAD_DRAFT);
        } else {
          const float p = a.target[(static_cast<size_t>(b) * (T + 1) + t) * V + x];
          const float q = a.draft ? a.draft[(static_cast<size_t>(b) * T + t) * V + x] : 1.f;
          ok = __fmul_rn(a.uniform[static_cast<size_t>(b) * (T + 1) + t], q) < p;
        }
      }
      const uint32_t refused = __ballot_sync(0xFFFFFFFFu, !ok);
      if (refused) {
        acc = t0 + __ffs(refused) - 1;
        break;
      }
    }
    if (lane == 0) {
      sh_acc = acc;
      sh_n = n;
    }
  }
  __syncthreads();
  const int acc = sh_acc, n = sh_n;
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
  const int mine = static_cast<int>(rank) * kVerifyWarps + warp;
  int token = -1;
  double W = 0.0;
  for (int attempt = 0; attempt < 2; ++attempt) {
    const int lo = min(V, mine * len), hi = min(V, lo + len);
    const double s = piece_sum<kVec>(row, lo, hi, lane);
    if (lane < static_cast<int>(ranks)) dsmem_store(&sums[mine], lane, s);
    v_cluster_sync();
    W = 0.0;                                            // every warp adds them in the same order
    for (int i = lane; i < static_cast<int>(ranks) * kVerifyWarps; i += 32) W += sums[i];
    W = warp_sum(W);
    if (W != 0.0 || (!row.q && row.drop < 0)) break;    // uniform over the cluster
    row.q = nullptr;                                    // p nowhere above q: sample from p itself
    row.drop = -1;
    v_cluster_sync();                                   // the sums have been read everywhere
  }
  const bool good = W > 0.0 && W < 1e300;               // finite (float sums reach 2^152 at most)
  const double r = static_cast<double>(a.uniform[static_cast<size_t>(b) * (T + 1) + T]) * W;
  double before = 0.0;
  const int piece = good ? find(sums, ranks * kVerifyWarps, r, before, lane) : -1;
  const bool owner = piece >= 0 ? piece / kVerifyWarps == static_cast<int>(rank) : rank == 0;
  if (owner) {                                          // uniform over the CTA
    if (piece >= 0) {
      // ---- the piece, cut once more over this CTA's warps
      const int lo = min(V, piece * len), hi = min(V, lo + len);
      const int sub = piece_len(hi - lo, kVerifyWarps);
      const int slo = min(hi, lo + warp * sub), shi = min(hi, slo + sub);
      const double s = piece_sum<kVec>(row, slo, shi, lane);
      if (lane == 0) part[warp] = s;
      __syncthreads();
      if (warp == 0) {
        double inner = 0.0;
        const int w = find(part, kVerifyWarps, r - before, inner, lane);
        // ---- and entry by entry: 32 at a time
        const int flo = min(hi, lo + max(w, 0) * sub), fhi = min(hi, flo + sub);
        double run = before + inner;
        int last = -1;
        for (int i0 = flo; i0 < fhi; i0 += 32) {
          const double v = i0 + lane < fhi ? static_cast<double>(weight_at(row, i0 + lane)) : 0.0;
          double in = v;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const double x = __shfl_up_sync(0xFFFFFFFFu, in, d);
            if (lane >= d) in += x;
          }
          const uint32_t hit = __ballot_sync(0xFFFFFFFFu, v > 0.0 && run + in > r);
          const uint32_t pos = __ballot_sync(0xFFFFFFFFu, v > 0.0);
          if (hit) {
            last = i0 + __ffs(hit) - 1;
            break;
          }
          if (pos) last = i0 + 31 - __clz(pos);
          run += __shfl_sync(0xFFFFFFFFu, in, 31);
        }
        token = last;
      }
    } else if (tid == 0) {
      report(a.status, ZF_DEV_BAD_PROBS);
    }
    if (warp == 0) {
      for (int t = lane; t <= T; t += 32)
        a.tokens[static_cast<size_t>(b) * (T + 1) + t] =
            t < acc ? a.tokens_in[static_cast<size_t>(b) * T + t] : t == acc ? token : -1;
      if (lane == 0) {
        a.accepted[b] = acc;
        if (a.out_lens) a.out_lens[b] = a.seq_lens[b] - (n - acc);
      }
    }
  }
  // no CTA reads another's shared memory after the last barrier (the sums were pushed), so none has to wait
}

template <bool kVec>
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
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<kVec>, a) == cudaSuccess ? ZF_OK : ZF_ERR_CUDA;
}

}  // namespace
}  // namespace zf

using namespace zf;

extern "C" zf_status zf_verify_drafts(int32_t batch, int32_t max_drafts, int32_t vocab, const float* target_probs,
                                      const float* draft_probs, const int32_t* draft_tokens, const int32_t* n_drafts,
                                      const float* uniform, int32_t* accepted, int32_t* tokens,
                                      const int32_t* seq_lens, int32_t* new_seq_lens, int32_t* status, void* stream) {
  if (batch < 0 || batch > ZF_MAX_BATCH || max_drafts < 1 || max_drafts > ZF_MAX_TOKENS || vocab < 1 ||
      vocab > ZF_MAX_VOCAB)
    return ZF_ERR_INVALID_ARGUMENT;
  if ((seq_lens == nullptr) != (new_seq_lens == nullptr)) return ZF_ERR_INVALID_ARGUMENT;
  if (batch == 0) return ZF_OK;
  if (!target_probs || !draft_tokens || !uniform || !accepted || !tokens) return ZF_ERR_INVALID_ARGUMENT;
  const void* all[] = {target_probs, draft_probs, draft_tokens, n_drafts, uniform, accepted, tokens, seq_lens,
                       new_seq_lens, status};
  for (const void* p : all)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return ZF_ERR_INVALID_ARGUMENT;
  VerifyArgs a{};
  a.target = target_probs;
  a.draft = draft_probs;
  a.tokens_in = draft_tokens;
  a.n_drafts = n_drafts;
  a.uniform = uniform;
  a.accepted = accepted;
  a.tokens = tokens;
  a.seq_lens = seq_lens;
  a.out_lens = new_seq_lens;
  a.status = status;
  a.batch = batch;
  a.T = max_drafts;
  a.vocab = vocab;
  // CTAs per request: enough to fill the 152 SMs with two CTAs each, at least 4096 entries per CTA.
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
      if (cudaFuncSetAttribute(verify_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
          cudaFuncSetAttribute(verify_kernel<false>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return ZF_ERR_CUDA;
      ready[dev] = true;
    }
  }
  const bool vec = vocab % 4 == 0 && aligned16(target_probs) && aligned16(draft_probs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return vec ? launch_verify<true>(a, ctas, s) : launch_verify<false>(a, ctas, s);
}
