// zf_map_tokens: block tables and slot maps from request lengths.
//
// need_b = ceil((len_b + new_b) / P), extra_b = max(0, need_b - held_b); exclusive prefix sums of new
// and extra in request order give each request its entries of the lists and its free pages; entry i
// of request b sits at position p = len_b + i, on page table[b][p / P] (or the free page that row
// entry is about to get), index p % P.
//
// A decode step is bound by latency (one launch, two dependent round trips), a batch of prompts by
// the 12 bytes it writes per token.  The first kernel is a single cluster of 1 or 8 CTAs, every one of
// which scans the whole batch (three loads per request) into its shared memory; the cluster barrier
// after that scan is what lets the outputs be the same arrays as the inputs.  The CTAs then share out
// the table entries and, for short lists, the list entries.  Long lists get a
// second, grid-wide kernel that works from the outputs of the first.  Either way a thread makes four
// entries at a time: one binary search over the list starts, one division, 16-byte stores.
#include <cuda_runtime.h>
#include <stdint.h>

#include <climits>
#include <mutex>

#include "zf_device.cuh"
#include "zf_host.h"

namespace zf {

namespace {

constexpr int kMapThreads = 1024;
constexpr int kMapPer = ZF_MAX_BATCH / kMapThreads;        // requests per thread of the scan

struct MapArgs {
  const int32_t* seq_lens;
  const int32_t* pages_held;
  const int32_t* new_tokens;
  int32_t* page_table;
  const int32_t* free_pages;
  const int32_t* free_pos;
  int32_t* out_lens;
  int32_t* out_held;
  int32_t* out_pos;
  int32_t* token_start;
  int32_t* page_ids;
  int32_t* positions;
  int32_t* seq_positions;
  int32_t* status;
  int32_t batch, page_size, max_pages, num_free, max_tokens;
  int32_t lists;               // whether the first kernel writes the list entries
};

// The largest b with start[b] <= i.
__device__ __forceinline__ int request_of(const int32_t* start, int batch, int i) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// List entries 4 c .. 4 c + 3: len(b) is request b's length before the call, page(b, j) its page j.
template <typename Len, typename Page>
__device__ __forceinline__ void write_entries(const MapArgs& a, const int32_t* start, int total, int c, Len&& len,
                                              Page&& page_of) {
  const int P = a.page_size, i0 = c * 4;
  int pid[4], pos[4], seq[4];
  int b = i0 < total ? request_of(start, a.batch, i0) : 0;
  int page = 0, in = -1, page_id = -1;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = i0 + e;
    if (i >= total) {
      pid[e] = pos[e] = seq[e] = -1;
      continue;
    }
    bool moved = e == 0, fresh = false;         // to another request; to another page
    while (start[b + 1] <= i) {
      ++b;
      moved = true;
    }
    const int p = len(b) + (i - start[b]);
    if (moved) {
      page = p / P;
      in = p - page * P;
      fresh = true;
    } else if (++in == P) {
      in = 0;
      ++page;
      fresh = true;
    }
    if (fresh) page_id = page_of(b, page);
    pid[e] = page_id;
    pos[e] = in;
    seq[e] = p;
  }
  if (i0 + 4 <= a.max_tokens) {
    *reinterpret_cast<int4*>(a.page_ids + i0) = make_int4(pid[0], pid[1], pid[2], pid[3]);
    *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    *reinterpret_cast<int4*>(a.seq_positions + i0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i0 + e < a.max_tokens) {
        a.page_ids[i0 + e] = pid[e];
        a.positions[i0 + e] = pos[e];
        a.seq_positions[i0 + e] = seq[e];
      }
    }
  }
}
__device__ __forceinline__ int entry_chunks(const MapArgs& a) {
  return static_cast<int>((static_cast<long long>(a.max_tokens) + 3) >> 2);
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

__global__ void __launch_bounds__(kMapThreads) map_kernel(const MapArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ long long warp_new[32], warp_extra[32];
  int32_t* start = sm;                          // [batch + 1] first list entry of each request
  int32_t* base = start + a.batch + 1;          // [batch] index of its first new page in free_pages
  int32_t* len = base + a.batch;                // [batch]
  int32_t* held = len + a.batch;                // [batch]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  allow_next_grid();
  wait_prior_grid();

  // ---- the batch: this thread's consecutive requests
  const int per = (a.batch + kMapThreads - 1) / kMapThreads;
  const int P = a.page_size;
  int nw[kMapPer], ex[kMapPer];
  long long sum_new = 0, sum_extra = 0;
  const int pos0 = *a.free_pos;
#pragma unroll
  for (int k = 0; k < kMapPer; ++k) {
    const int b = tid * per + k;
    nw[k] = ex[k] = 0;
    if (k < per && b < a.batch) {
      const int L = a.seq_lens[b], h = a.pages_held[b], n = a.new_tokens[b];
      len[b] = L;
      held[b] = h;
      const long long cap = static_cast<long long>(a.max_pages) * P;
      const bool ok = L >= 0 && n >= 0 && h >= 0 && h <= a.max_pages && L <= static_cast<long long>(h) * P &&
                      static_cast<long long>(L) + n <= cap;
      if (ok) {
        nw[k] = n;
        ex[k] = max(0, static_cast<int>((static_cast<uint32_t>(L) + n + P - 1u) / P) - h);    // (L + n may be near 2^31)
        sum_new += nw[k];
        sum_extra += ex[k];
      } else if (rank == 0) {
        report(a.status, ZF_DEV_BAD_SEQ_LEN);
      }
    }
  }
  // ---- prefix sums over the threads (64 bits: a refused call's totals may not fit 32)
  long long in_new = sum_new, in_extra = sum_extra;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, in_new, d), y = __shfl_up_sync(0xFFFFFFFFu, in_extra, d);
    if (lane >= d) {
      in_new += x;
      in_extra += y;
    }
  }
  if (lane == 31) {
    warp_new[warp] = in_new;
    warp_extra[warp] = in_extra;
  }
  __syncthreads();
  long long off_new = 0, off_extra = 0, total_new = 0, total_extra = 0;
  const int used = ((a.batch + max(per, 1) - 1) / max(per, 1) + 31) / 32;      // warps that hold requests
#pragma unroll 4
  for (int w = 0; w < used; ++w) {
    const long long x = warp_new[w], y = warp_extra[w];
    if (w < warp) {
      off_new += x;
      off_extra += y;
    }
    total_new += x;
    total_extra += y;
  }
  const bool fits = pos0 >= 0 && total_new <= a.max_tokens && total_extra + pos0 <= a.num_free;
  if (!fits && rank == 0 && tid == 0) report(a.status, ZF_DEV_CAPACITY);
  long long at_new = off_new + in_new - sum_new, at_extra = pos0 + off_extra + in_extra - sum_extra;
#pragma unroll
  for (int k = 0; k < kMapPer; ++k) {
    const int b = tid * per + k;
    if (k < per && b < a.batch) {
      start[b] = fits ? static_cast<int>(at_new) : 0;
      base[b] = fits ? static_cast<int>(at_extra) : 0;
      at_new += nw[k];
      at_extra += ex[k];
    }
  }
  if (tid == 0) start[a.batch] = fits ? static_cast<int>(total_new) : 0;
  __syncthreads();
  // every CTA has read the inputs: from here on they may be overwritten
  cluster_sync();

  // ---- per request: lengths, pages, list starts (CTA 0)
  if (rank == 0) {
#pragma unroll
    for (int k = 0; k < kMapPer; ++k) {
      const int b = tid * per + k;
      if (k < per && b < a.batch) {
        a.out_lens[b] = len[b] + (fits ? nw[k] : 0);
        a.out_held[b] = held[b] + (fits ? ex[k] : 0);
        a.token_start[b] = start[b];
      }
    }
    if (tid == 0) {
      a.token_start[a.batch] = start[a.batch];
      *a.out_pos = pos0 + (fits ? static_cast<int>(total_extra) : 0);
    }
  }
  const int total = start[a.batch];

  // ---- list entries.  A page past those held is read from the free list, not from the table, whose
  // new entries are being written below at the same time.
  if (a.lists) {
    const int chunks = entry_chunks(a);
    for (int c = rank * kMapThreads + tid; c < chunks; c += ranks * kMapThreads)
      write_entries(a, start, total, c, [&](int b) { return len[b]; },
                    [&](int b, int j) {
                      return j < held[b] ? a.page_table[static_cast<size_t>(b) * a.max_pages + j]
                                         : a.free_pages[base[b] + j - held[b]];
                    });
  }

  // ---- new table entries: one thread each, whatever requests they belong to
  if (fits) {
    const long long end = pos0 + total_extra;
    for (long long k = static_cast<long long>(pos0) + rank * kMapThreads + tid; k < end; k += ranks * kMapThreads) {
      const int j = static_cast<int>(k);
      const int b = request_of(base, a.batch, j);
      a.page_table[static_cast<size_t>(b) * a.max_pages + held[b] + (j - base[b])] = a.free_pages[j];
    }
  }
}

// List entries of a long list, from what the first kernel wrote.
constexpr int kListThreads = 256;
__global__ void __launch_bounds__(kListThreads) list_kernel(const MapArgs a) {
  extern __shared__ int32_t start[];               // [batch + 1]
  allow_next_grid();
  wait_prior_grid();
  for (int i = threadIdx.x; i <= a.batch; i += kListThreads) start[i] = a.token_start[i];
  __syncthreads();
  const int total = start[a.batch], chunks = entry_chunks(a);
  for (long long c = static_cast<long long>(blockIdx.x) * kListThreads + threadIdx.x; c < chunks;
       c += static_cast<long long>(gridDim.x) * kListThreads)
    write_entries(a, start, total, static_cast<int>(c),
                  [&](int b) { return a.out_lens[b] - (start[b + 1] - start[b]); },
                  [&](int b, int j) { return a.page_table[static_cast<size_t>(b) * a.max_pages + j]; });
}

}  // namespace
}  // namespace zf

using namespace zf;

extern "C" zf_status zf_map_tokens(int32_t batch, int32_t page_size, int32_t max_pages, const int32_t* seq_lens,
                                   const int32_t* pages_held, const int32_t* new_tokens, int32_t* page_table,
                                   const int32_t* free_pages, int32_t num_free, const int32_t* free_pos,
                                   int32_t* new_seq_lens, int32_t* new_pages_held, int32_t* new_free_pos,
                                   int32_t* token_start, int32_t* page_ids, int32_t* positions,
                                   int32_t* seq_positions, int32_t max_tokens, int32_t* status, void* stream) {
  if (batch < 0 || batch > ZF_MAX_BATCH || max_pages < 1 || num_free < 0 || max_tokens < 0 ||
      max_tokens > (1 << 30))
    return ZF_ERR_INVALID_ARGUMENT;
  if (page_size < ZF_BLOCK_TOKENS || page_size % ZF_BLOCK_TOKENS) return ZF_ERR_INVALID_ARGUMENT;
  if (page_size > ZF_MAX_PAGE_SIZE) return ZF_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size >= INT_MAX) return ZF_ERR_INVALID_ARGUMENT;
  const void* always[] = {free_pos, new_free_pos, token_start};
  for (const void* p : always)
    if (!p || (reinterpret_cast<uintptr_t>(p) & 3u)) return ZF_ERR_INVALID_ARGUMENT;
  const void* per_request[] = {seq_lens, pages_held, new_tokens, page_table, new_seq_lens, new_pages_held};
  for (const void* p : per_request)
    if ((batch > 0 && !p) || (reinterpret_cast<uintptr_t>(p) & 3u)) return ZF_ERR_INVALID_ARGUMENT;
  if ((num_free > 0 && !free_pages) || (reinterpret_cast<uintptr_t>(free_pages) & 3u) ||
      (reinterpret_cast<uintptr_t>(status) & 3u))
    return ZF_ERR_INVALID_ARGUMENT;
  const void* lists[] = {page_ids, positions, seq_positions};
  for (const void* p : lists)
    if (max_tokens > 0 && (!p || !aligned16(p))) return ZF_ERR_INVALID_ARGUMENT;
  MapArgs a{};
  a.seq_lens = seq_lens;
  a.pages_held = pages_held;
  a.new_tokens = new_tokens;
  a.page_table = page_table;
  a.free_pages = free_pages;
  a.free_pos = free_pos;
  a.out_lens = new_seq_lens;
  a.out_held = new_pages_held;
  a.out_pos = new_free_pos;
  a.token_start = token_start;
  a.page_ids = page_ids;
  a.positions = positions;
  a.seq_positions = seq_positions;
  a.status = status;
  a.batch = batch;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.num_free = num_free;
  a.max_tokens = max_tokens;
  // Lists of up to kShortList entries are written by the first kernel, by one CTA up to 4096 entries
  // (one pass of its threads), else by a cluster of 8.
  constexpr int kShortList = 32768;
  const int ctas = max_tokens <= 4096 ? 1 : 8;
  a.lists = max_tokens <= kShortList ? 1 : 0;
  const size_t smem = (static_cast<size_t>(batch) * 4 + 1) * 4;
  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZF_ERR_CUDA;
  if (dev < 0 || dev >= 64) return ZF_ERR_UNSUPPORTED;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      const int most = (ZF_MAX_BATCH * 4 + 1) * 4;
      if (cudaFuncSetAttribute(map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
        return ZF_ERR_CUDA;
      ready[dev] = true;
    }
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kMapThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;       // (one CTA: a plain launch, 2 us less on the host)
  if (cudaLaunchKernelEx(&cfg, map_kernel, a) != cudaSuccess) return ZF_ERR_CUDA;
  if (a.lists) return ZF_OK;
  const long long blocks = ((static_cast<long long>(max_tokens) + 3) / 4 + kListThreads - 1) / kListThreads;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < 1216 ? blocks : 1216));       // 152 SMs x 8 resident CTAs
  cfg.blockDim = dim3(kListThreads);
  cfg.dynamicSmemBytes = (static_cast<size_t>(batch) + 1) * 4;
  cfg.numAttrs = 1;                                                               // no cluster
  return cudaLaunchKernelEx(&cfg, list_kernel, a) == cudaSuccess ? ZF_OK : ZF_ERR_CUDA;
}
