// Pages of a paged cache shared, given back and moved on the GPU: zf_fork_requests, zf_release_requests,
// zf_compact_pages and zf_q4_copy_pages.
//
// Who holds a page is read from the page table (rows' first pages_held entries) whenever it is needed: there are no
// holder counts that could fall out of step with it.
//
// The first three are bound by latency: a few dependent passes over lists of a few hundred KB that lie in L2.
// Each is one cluster of CTAs (1 or 16), whose barrier separates the passes and, as in zf_map_tokens, lets
// outputs be the same arrays as inputs.  64 requests of 1024 tokens, 4096 entries: fork 5.9 us, release 9.4, compact 10.5
// (three quarters of the entries held), of which a launch and the first dependent loads are some 4.  The copy is bound by its bytes, read and written once:
// 81 MB of pages in 28.0 us, 5.8 TB/s (6.7 is a plain copy's rate).
#include <cuda_runtime.h>
#include <stdint.h>

#include <climits>
#include <initializer_list>
#include <mutex>

#include "zf_device.cuh"
#include "zf_host.h"
#include "zf_q4.cuh"

namespace zf {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 16;
constexpr int kPer = ZF_MAX_BATCH / kThreads;        // requests per thread of a scan
constexpr int kPiece = 256;                          // table entries that a warp takes at a time

__device__ __forceinline__ uint32_t rank_in_cluster() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t ranks_of_cluster() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Store into CTA `rank`'s copy of a shared variable.
__device__ __forceinline__ void store_to(int* p, uint32_t rank, int v) {
  uint32_t addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Sum over the block's threads before this one; total: of all.  sh: [kWarps], free again after the call's barriers.
__device__ __forceinline__ int block_scan(int v, int* sh, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int in = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, in, d);
    if (lane >= d) in += x;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = in;
  __syncthreads();
  const int w = sh[lane];
  int before = lane < warp ? w : 0, all = w;
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  total = __reduce_add_sync(0xFFFFFFFFu, all);
  return before + in - v;
}

// One value of every CTA of the cluster: the sum of those before this one; total: of all.  sh: [kCluster], used once.
__device__ __forceinline__ int cluster_scan(int v, int* sh, uint32_t rank, uint32_t ranks, int& total) {
  if (threadIdx.x < ranks) store_to(&sh[rank], threadIdx.x, v);
  cluster_sync();
  int before = 0;
  total = 0;
  for (uint32_t k = 0; k < ranks; ++k) {
    const int x = sh[k];
    if (k < rank) before += x;
    total += x;
  }
  return before;
}

// f(row, entry, page) for the first held[row] entries of every row: pieces of kPiece entries, a warp each, over the
// whole cluster.
template <typename F>
__device__ __forceinline__ void for_pages(const int32_t* table, int batch, int max_pages, const int32_t* held, uint32_t rank,
                                          uint32_t ranks, F&& f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pieces = (max_pages + kPiece - 1) / kPiece;
  const long long items = static_cast<long long>(batch) * pieces;
  for (long long k = rank * kWarps + warp; k < items; k += ranks * kWarps) {
    const int b = static_cast<int>(k / pieces), j0 = static_cast<int>(k - static_cast<long long>(b) * pieces) * kPiece;
    const int n = held[b];
    if (j0 >= n) continue;
    const int32_t* row = table + static_cast<size_t>(b) * max_pages;
    int page[kPiece / 32];
#pragma unroll
    for (int e = 0; e < kPiece / 32; ++e) {
      const int j = j0 + 32 * e + lane;
      page[e] = j < n ? row[j] : 0;
    }
#pragma unroll
    for (int e = 0; e < kPiece / 32; ++e) {
      const int j = j0 + 32 * e + lane;
      if (j < n) f(b, j, page[e]);
    }
  }
}

// ------------------------------------------------------------------------------------------- fork
struct ForkArgs {
  const int32_t* seq_lens;
  const int32_t* pages_held;
  const int32_t* src;
  const int32_t* dst;
  int32_t* page_table;
  const int32_t* free_pages;
  const int32_t* free_pos;
  int32_t* out_lens;
  int32_t* out_held;
  int32_t* out_pos;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* status;
  int32_t batch, n, page_size, max_pages, num_free;
};

// Every CTA works out all forks (a thread four at a time) into its shared memory; then the CTAs share out the rows.
__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ int sh[kWarps];
  int32_t* by_row = sm;                          // [batch] the fork that fills this row; INT_MAX: none
  int32_t* from = by_row + a.batch;              // [n] source row; -1: refused
  int32_t* len = from + a.n;                     // [n] tokens
  int32_t* tail = len + a.n;                     // [n] index in free_pages of the tail's copy; -1: no tail
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = rank_in_cluster(), ranks = ranks_of_cluster();
  allow_next_grid();
  wait_prior_grid();
  for (int b = tid; b < a.batch; b += kThreads) by_row[b] = INT_MAX;
  __syncthreads();
  const int pos0 = *a.free_pos, P = a.page_size;
  for (int i = tid; i < a.n; i += kThreads) {
    const int d = a.dst[i];
    if (d >= 0 && d < a.batch) atomicMin(&by_row[d], i);         // the first that names a row has it
  }
  __syncthreads();
  int need[kPer], sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = tid * kPer + k;
    need[k] = 0;
    if (i < a.n) {
      const int s = a.src[i], d = a.dst[i];
      bool ok = s >= 0 && s < a.batch && d >= 0 && d < a.batch && s != d;
      int L = 0;
      if (ok) {
        const int h = a.pages_held[s];
        L = a.seq_lens[s];
        ok = L >= 0 && h >= 0 && h <= a.max_pages && L <= static_cast<long long>(h) * P && a.pages_held[d] == 0 &&
             a.seq_lens[d] == 0 && by_row[d] == i;
      }
      if (!ok && rank == 0) report(a.status, ZF_DEV_BAD_FORK);
      from[i] = ok ? s : -1;
      len[i] = L;
      need[k] = ok && L % P != 0;
      sum += need[k];
    }
  }
  int total;
  int at = block_scan(sum, sh, total);
  const bool fits = pos0 >= 0 && static_cast<long long>(pos0) + total <= a.num_free;
  if (!fits && rank == 0 && tid == 0) report(a.status, ZF_DEV_CAPACITY);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = tid * kPer + k;
    if (i < a.n) {
      tail[i] = need[k] ? pos0 + at : -1;
      at += need[k];
      if (!fits) from[i] = -1;
    }
  }
  __syncthreads();
  cluster_sync();                                // all inputs are read: they may be overwritten from here on

  if (rank == 0) {
    for (int b = tid; b < a.batch; b += kThreads) {
      const int i = by_row[b];
      const bool filled = i < a.n && from[i] >= 0;
      a.out_lens[b] = filled ? len[i] : a.seq_lens[b];
      a.out_held[b] = filled ? len[i] / P + (tail[i] >= 0) : a.pages_held[b];
    }
    if (tid == 0) *a.out_pos = pos0 + (fits ? total : 0);
  }
  // ---- table rows: full pages shared, the tail's page new
  const int pieces = (a.max_pages + kPiece - 1) / kPiece;
  const long long items = static_cast<long long>(a.n) * pieces;
  for (long long k = rank * kWarps + warp; k < items; k += ranks * kWarps) {
    const int i = static_cast<int>(k / pieces), j0 = static_cast<int>(k - static_cast<long long>(i) * pieces) * kPiece;
    const int s = from[i];
    if (s < 0) {
      if (j0 == 0 && lane == 0) a.copy_src[i] = a.copy_dst[i] = -1;
      continue;
    }
    const int full = len[i] / P;
    const int32_t* in = a.page_table + static_cast<size_t>(s) * a.max_pages;
    int32_t* out = a.page_table + static_cast<size_t>(a.dst[i]) * a.max_pages;
    int page[kPiece / 32];
#pragma unroll
    for (int e = 0; e < kPiece / 32; ++e) {
      const int j = j0 + 32 * e + lane;
      page[e] = j < full ? in[j] : 0;
    }
#pragma unroll
    for (int e = 0; e < kPiece / 32; ++e) {
      const int j = j0 + 32 * e + lane;
      if (j < full) out[j] = page[e];
    }
    if (j0 == 0 && lane == 0) {
      const bool has = tail[i] >= 0;
      const int fresh = has ? a.free_pages[tail[i]] : -1;
      a.copy_src[i] = has ? in[full] : -1;
      a.copy_dst[i] = fresh;
      if (has) out[full] = fresh;
    }
  }
}

// ---------------------------------------------------------------------------------------- release
struct ReleaseArgs {
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* pages_held;
  const int32_t* release;
  int32_t* free_pages;
  const int32_t* free_pos;
  int32_t* out_lens;
  int32_t* out_held;
  int32_t* out_pos;
  int32_t* claim;                                // [num_pages]
  int32_t* status;
  int32_t batch, max_pages, num_pages, num_free;
};

// The mentions of pages by released rows are numbered in row order.  claim[page] becomes the smallest number that
// mentions it, or -1 when a row that stays does; the mention that finds its own number there frees the page.  Only
// entries of pages that are mentioned are touched.
__global__ void __launch_bounds__(kThreads) release_kernel(const ReleaseArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ int sh[kWarps], shc[kCluster];
  int32_t* held = sm;                            // [batch] pages of the row
  int32_t* base = held + a.batch;                // [batch + 1] number of its first mention; rows that stay: the next one's
  const int tid = threadIdx.x;
  const uint32_t rank = rank_in_cluster(), ranks = ranks_of_cluster();
  allow_next_grid();
  wait_prior_grid();
  const int pos0 = *a.free_pos;
  int mine[kPer], sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = tid * kPer + k;
    mine[k] = 0;
    if (b < a.batch) {
      int h = a.pages_held[b];
      if (h < 0 || h > a.max_pages) {
        if (rank == 0) report(a.status, ZF_DEV_BAD_SEQ_LEN);
        h = min(max(h, 0), a.max_pages);
      }
      held[b] = h;
      mine[k] = a.release[b] != 0 ? h : 0;
      sum += mine[k];
    }
  }
  int mentions;
  int at = block_scan(sum, sh, mentions);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = tid * kPer + k;
    if (b < a.batch) base[b] = at;
    at += mine[k];
  }
  if (tid == 0) base[a.batch] = mentions;
  __syncthreads();
  auto released = [&](int b) { return base[b + 1] > base[b]; };      // (a released row without pages mentions none)
  for_pages(a.page_table, a.batch, a.max_pages, held, rank, ranks, [&](int, int, int page) {
    if (page >= 0 && page < a.num_pages) a.claim[page] = INT_MAX;
    else report(a.status, ZF_DEV_BAD_PAGE_ID);
  });
  cluster_sync();
  for_pages(a.page_table, a.batch, a.max_pages, held, rank, ranks, [&](int b, int j, int page) {
    if (page >= 0 && page < a.num_pages) atomicMin(&a.claim[page], released(b) ? base[b] + j : -1);
  });
  cluster_sync();

  // ---- this CTA's mentions: how many free a page, then where they go
  const int per = (mentions + static_cast<int>(ranks) - 1) / static_cast<int>(ranks);
  const int lo = min(mentions, static_cast<int>(rank) * per), hi = min(mentions, lo + per);
  auto freed = [&](int e) {                      // the page that mention e frees, or -1
    int l = 0, h = a.batch;                      // base[l] <= e < base[h]
    while (h - l > 1) {
      const int mid = (l + h) >> 1;
      if (base[mid] <= e) l = mid; else h = mid;
    }
    const int page = a.page_table[static_cast<size_t>(l) * a.max_pages + (e - base[l])];
    return page >= 0 && page < a.num_pages && ld_relaxed(&a.claim[page]) == e ? page : -1;
  };
  int count = 0;
  for (int e = lo + tid; e < hi; e += kThreads) count += freed(e) >= 0;
  int here;
  block_scan(count, sh, here);
  int total;
  const int before = cluster_scan(here, shc, rank, ranks, total);
  const bool fits = pos0 <= a.num_free && total <= pos0;
  if (!fits && rank == 0 && tid == 0) report(a.status, ZF_DEV_CAPACITY);
  if (fits) {
    int to = pos0 - total + before;
    for (int e0 = lo; e0 < hi; e0 += kThreads) {
      const int page = e0 + tid < hi ? freed(e0 + tid) : -1;
      int n;
      const int k = block_scan(page >= 0, sh, n);
      if (page >= 0) a.free_pages[to + k] = page;
      to += n;
    }
  }
  if (rank == 0) {
    for (int b = tid; b < a.batch; b += kThreads) {
      const bool gone = fits && a.release[b] != 0;
      a.out_lens[b] = gone ? 0 : a.seq_lens[b];
      a.out_held[b] = gone ? 0 : a.pages_held[b];
    }
    if (tid == 0) *a.out_pos = fits ? pos0 - total : pos0;
  }
}

// ---------------------------------------------------------------------------------------- compact
struct CompactArgs {
  const int32_t* page_table;
  const int32_t* pages_held;
  int32_t* out_table;
  int32_t* free_pages;                           // [num_pages]
  int32_t* free_pos;
  int32_t* copy_src;                             // [num_pages / 2]
  int32_t* copy_dst;
  uint32_t* used;                                // [words] bit per page
  int32_t* to;                                   // [num_pages] where a page that moves goes
  int32_t* status;
  int32_t batch, max_pages, num_pages;
};

// With n pages in use, those with ids from n on move to the unused ids below n, both in ascending order.
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
  extern __shared__ int32_t held[];              // [batch]
  __shared__ int sh[kWarps], shc[4][kCluster];
  const int tid = threadIdx.x;
  const uint32_t rank = rank_in_cluster(), ranks = ranks_of_cluster();
  allow_next_grid();
  wait_prior_grid();
  const int words = (a.num_pages + 31) / 32;
  const int step = static_cast<int>(ranks) * kThreads, first = static_cast<int>(rank) * kThreads + tid;
  for (int w = first; w < words; w += step) a.used[w] = 0;
  for (int b = tid; b < a.batch; b += kThreads) {
    int h = a.pages_held[b];
    if (h < 0 || h > a.max_pages) {
      if (rank == 0) report(a.status, ZF_DEV_BAD_SEQ_LEN);
      h = min(max(h, 0), a.max_pages);
    }
    held[b] = h;
  }
  __syncthreads();
  cluster_sync();
  for_pages(a.page_table, a.batch, a.max_pages, held, rank, ranks, [&](int, int, int page) {
    if (page >= 0 && page < a.num_pages) atomicOr(&a.used[page >> 5], 1u << (page & 31));
    else report(a.status, ZF_DEV_BAD_PAGE_ID);
  });
  cluster_sync();

  // ---- this CTA's words, a run of consecutive ones per thread
  const int per_cta = (words + static_cast<int>(ranks) - 1) / static_cast<int>(ranks);
  const int lo = min(words, static_cast<int>(rank) * per_cta), hi = min(words, lo + per_cta);
  const int per = (hi - lo + kThreads - 1) / kThreads;
  const int w0 = min(hi, lo + tid * per), w1 = min(hi, w0 + per);
  auto word = [&](int w) { return static_cast<uint32_t>(ld_relaxed(reinterpret_cast<const int32_t*>(a.used) + w)); };
  int count = 0, here, n;
  for (int w = w0; w < w1; ++w) count += __popc(word(w));
  block_scan(count, sh, here);
  cluster_scan(here, shc[0], rank, ranks, n);
  // the pages of word w that move, and the places that they can go to
  auto below = [&](int w) {                      // bits of word w with ids below n
    const long long k = static_cast<long long>(n) - 32ll * w;
    return k <= 0 ? 0u : k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u;
  };
  int moves = 0, holes = 0;
  for (int w = w0; w < w1; ++w) {
    const uint32_t u = word(w), m = below(w);
    moves += __popc(u & ~m);
    holes += __popc(~u & m);
  }
  int here_m, here_h, total;
  int at_m = block_scan(moves, sh, here_m), at_h = block_scan(holes, sh, here_h);
  at_m += cluster_scan(here_m, shc[1], rank, ranks, total);
  int same;
  at_h += cluster_scan(here_h, shc[2], rank, ranks, same);
  for (int w = w0; w < w1; ++w) {
    const uint32_t u = word(w), m = below(w);
    for (uint32_t x = u & ~m; x; x &= x - 1) a.copy_src[at_m++] = 32 * w + __ffs(x) - 1;
    for (uint32_t x = ~u & m; x; x &= x - 1) a.copy_dst[at_h++] = 32 * w + __ffs(x) - 1;
  }
  for (int k = total + first; k < a.num_pages / 2; k += step) a.copy_src[k] = a.copy_dst[k] = -1;
  for (int k = first; k < a.num_pages; k += step) a.free_pages[k] = k < n ? -1 : k;
  if (first == 0) *a.free_pos = n;
  cluster_sync();
  for (int k = first; k < total; k += step) a.to[ld_relaxed(&a.copy_src[k])] = ld_relaxed(&a.copy_dst[k]);
  cluster_sync();
  const long long entries = static_cast<long long>(a.batch) * a.max_pages;
  for (long long k = first; k < entries; k += step) {
    const int b = static_cast<int>(k / a.max_pages), j = static_cast<int>(k - static_cast<long long>(b) * a.max_pages);
    const int page = a.page_table[k];
    a.out_table[k] = j < held[b] && page >= n && page < a.num_pages ? ld_relaxed(&a.to[page]) : page;
  }
}

// ------------------------------------------------------------------------------------------- copy
constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = kCopyThreads * 64;    // four 16-byte loads per thread in flight

struct CopyArgs {
  uint8_t* records;
  const int32_t* src;
  const int32_t* dst;
  int32_t* status;
  size_t page_bytes;
  int32_t n, num_pages, chunks;                  // chunks: pieces of kCopyBytes of a page
};

// A CTA looks at 256 pieces at once (its own, a grid apart), so that lists which are mostly padding cost little, and
// copies those that are pages one after another.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyArgs a) {
  __shared__ int sh_from[kCopyThreads], sh_to[kCopyThreads], sh_piece[kCopyThreads], sh_n;
  const int tid = threadIdx.x;
  allow_next_grid();
  wait_prior_grid();
  const long long items = static_cast<long long>(a.n) * a.chunks;
  for (long long k0 = blockIdx.x; k0 < items; k0 += static_cast<long long>(gridDim.x) * kCopyThreads) {
    if (tid == 0) sh_n = 0;
    __syncthreads();
    const long long k = k0 + static_cast<long long>(tid) * gridDim.x;
    if (k < items) {
      const int i = static_cast<int>(k / a.chunks);
      const int s = a.src[i], d = a.dst[i];
      const bool in = s >= 0 && s < a.num_pages && d >= 0 && d < a.num_pages;
      if (in && s != d) {
        const int at = atomicAdd(&sh_n, 1);      // (their order does not matter)
        sh_from[at] = s;
        sh_to[at] = d;
        sh_piece[at] = static_cast<int>(k - static_cast<long long>(i) * a.chunks);
      } else if (!in && !(s == -1 && d == -1)) {
        report(a.status, ZF_DEV_BAD_PAGE_ID);
      }
    }
    __syncthreads();
    const int n = sh_n;
    for (int e = 0; e < n; ++e) {
      const size_t first = static_cast<size_t>(sh_piece[e]) * kCopyBytes;
      const uint8_t* from = a.records + static_cast<size_t>(sh_from[e]) * a.page_bytes + first;
      uint8_t* to = a.records + static_cast<size_t>(sh_to[e]) * a.page_bytes + first;
      const int bytes = static_cast<int>(min(a.page_bytes - first, static_cast<size_t>(kCopyBytes)));
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int x = (j * kCopyThreads + tid) * 16;
        if (x < bytes) v[j] = *reinterpret_cast<const uint4*>(from + x);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int x = (j * kCopyThreads + tid) * 16;
        if (x < bytes) *reinterpret_cast<uint4*>(to + x) = v[j];
      }
    }
    __syncthreads();
  }
}

// Launch of one cluster of `ctas` (1: a plain launch) with `smem` bytes.
template <typename Kernel, typename Args>
zf_status launch_cluster(Kernel kernel, int which, int ctas, size_t smem, size_t most, cudaStream_t s, const Args& args) {
  static std::mutex mu;
  static bool ready[64][3] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZF_ERR_CUDA;
  if (dev < 0 || dev >= 64) return ZF_ERR_UNSUPPORTED;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev][which]) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most)) != cudaSuccess)
        return ZF_ERR_CUDA;
      ready[dev][which] = true;
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
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess ? ZF_OK : ZF_ERR_CUDA;
}

bool words_ok(std::initializer_list<const void*> needed, std::initializer_list<const void*> optional = {}) {
  for (const void* p : needed)
    if (!p || (reinterpret_cast<uintptr_t>(p) & 3u)) return false;
  for (const void* p : optional)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return false;
  return true;
}
bool table_ok(int batch, int max_pages) { return batch >= 0 && batch <= ZF_MAX_BATCH && max_pages >= 1; }
bool pool_ok(int num_pages) { return num_pages >= 0 && num_pages <= INT_MAX - (1 << 20); }
// CTAs for passes over a table of so many entries.  Release + compaction, us, with all entries held, one CTA and 16: 2048
// entries 9.6 + 8.1 and 10.1 + 11.1; 4096 14.7 + 10.1 and 10.4 + 11.5; 8192 24.8 + 13.6 and 12.9 + 11.7; 16384 46 + 23 and
// 14 + 13; 65536 190 + 83 and 20 + 16; 262144 784 + 298 and 59 + 34 (8 CTAs: 13 + 11 at 8192, 108 + 56 at 262144).  A table
// in use has room that is not held, so the border lies at twice the entries where the two are alike.
int ctas_for(long long entries) { return entries <= 8192 ? 1 : kCluster; }

}  // namespace
}  // namespace zf

using namespace zf;

extern "C" zf_status zf_fork_requests(int32_t batch, int32_t page_size, int32_t max_pages, const int32_t* seq_lens,
                                      const int32_t* pages_held, const int32_t* src, const int32_t* dst, int32_t n,
                                      int32_t* page_table, const int32_t* free_pages, int32_t num_free,
                                      const int32_t* free_pos, int32_t* new_seq_lens, int32_t* new_pages_held,
                                      int32_t* new_free_pos, int32_t* copy_src, int32_t* copy_dst, int32_t* status,
                                      void* stream) {
  if (!table_ok(batch, max_pages) || n < 0 || n > ZF_MAX_BATCH || num_free < 0) return ZF_ERR_INVALID_ARGUMENT;
  if (page_size < ZF_BLOCK_TOKENS || page_size % ZF_BLOCK_TOKENS) return ZF_ERR_INVALID_ARGUMENT;
  if (page_size > ZF_MAX_PAGE_SIZE) return ZF_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size >= INT_MAX) return ZF_ERR_INVALID_ARGUMENT;
  if (!words_ok({free_pos, new_free_pos}, {status, free_pages}) || (num_free > 0 && !free_pages)) return ZF_ERR_INVALID_ARGUMENT;
  if (!(batch > 0 ? words_ok({seq_lens, pages_held, page_table, new_seq_lens, new_pages_held}) : true) ||
      !(n > 0 ? words_ok({src, dst, copy_src, copy_dst}) : true))
    return ZF_ERR_INVALID_ARGUMENT;
  ForkArgs a{};
  a.seq_lens = seq_lens;
  a.pages_held = pages_held;
  a.src = src;
  a.dst = dst;
  a.page_table = page_table;
  a.free_pages = free_pages;
  a.free_pos = free_pos;
  a.out_lens = new_seq_lens;
  a.out_held = new_pages_held;
  a.out_pos = new_free_pos;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.status = status;
  a.batch = batch;
  a.n = n;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.num_free = num_free;
  const size_t smem = (static_cast<size_t>(batch) + 3 * static_cast<size_t>(n)) * 4;
  return launch_cluster(fork_kernel, 0, ctas_for(static_cast<long long>(n) * max_pages), smem, ZF_MAX_BATCH * 16,
                        static_cast<cudaStream_t>(stream), a);
}

extern "C" size_t zf_release_requests_workspace_size(int32_t num_pages) {
  return pool_ok(num_pages) ? (static_cast<size_t>(num_pages) * 4 + 255) & ~static_cast<size_t>(255) : 0;
}

extern "C" zf_status zf_release_requests(int32_t batch, int32_t max_pages, int32_t num_pages, const int32_t* page_table,
                                         const int32_t* seq_lens, const int32_t* pages_held, const int32_t* release,
                                         int32_t* free_pages, int32_t num_free, const int32_t* free_pos,
                                         int32_t* new_seq_lens, int32_t* new_pages_held, int32_t* new_free_pos,
                                         int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  if (!table_ok(batch, max_pages) || !pool_ok(num_pages) || num_free < 0) return ZF_ERR_INVALID_ARGUMENT;
  // mentions of pages are numbered with 32 bits
  if (static_cast<long long>(batch) * max_pages > (1ll << 30)) return ZF_ERR_UNSUPPORTED;
  if (!words_ok({free_pos, new_free_pos}, {status, free_pages}) || (num_free > 0 && !free_pages)) return ZF_ERR_INVALID_ARGUMENT;
  if (batch > 0 && !words_ok({page_table, seq_lens, pages_held, release, new_seq_lens, new_pages_held}))
    return ZF_ERR_INVALID_ARGUMENT;
  if (num_pages > 0 && (!workspace || !aligned16(workspace))) return ZF_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < zf_release_requests_workspace_size(num_pages)) return ZF_ERR_WORKSPACE_TOO_SMALL;
  ReleaseArgs a{};
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.pages_held = pages_held;
  a.release = release;
  a.free_pages = free_pages;
  a.free_pos = free_pos;
  a.out_lens = new_seq_lens;
  a.out_held = new_pages_held;
  a.out_pos = new_free_pos;
  a.claim = static_cast<int32_t*>(workspace);
  a.status = status;
  a.batch = batch;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.num_free = num_free;
  const size_t smem = (2 * static_cast<size_t>(batch) + 1) * 4;
  return launch_cluster(release_kernel, 1, ctas_for(static_cast<long long>(batch) * max_pages), smem,
                        (2 * ZF_MAX_BATCH + 1) * 4, static_cast<cudaStream_t>(stream), a);
}

extern "C" size_t zf_compact_pages_workspace_size(int32_t num_pages) {
  if (!pool_ok(num_pages)) return 0;
  const size_t words = (static_cast<size_t>(num_pages) + 31) / 32;
  return ((words + static_cast<size_t>(num_pages)) * 4 + 255) & ~static_cast<size_t>(255);
}

extern "C" zf_status zf_compact_pages(int32_t batch, int32_t max_pages, int32_t num_pages, const int32_t* page_table,
                                      const int32_t* pages_held, int32_t* new_page_table, int32_t* free_pages,
                                      int32_t* free_pos, int32_t* copy_src, int32_t* copy_dst, int32_t* status,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!table_ok(batch, max_pages) || !pool_ok(num_pages)) return ZF_ERR_INVALID_ARGUMENT;
  // a row's entries are counted with 32 bits, and in pieces of kPiece
  if (max_pages > (1 << 30)) return ZF_ERR_UNSUPPORTED;
  if (!words_ok({free_pos}, {status})) return ZF_ERR_INVALID_ARGUMENT;
  if (batch > 0 && !words_ok({page_table, pages_held, new_page_table})) return ZF_ERR_INVALID_ARGUMENT;
  if (num_pages > 0 && (!words_ok({free_pages}) || !workspace || !aligned16(workspace))) return ZF_ERR_INVALID_ARGUMENT;
  if (num_pages > 1 && !words_ok({copy_src, copy_dst})) return ZF_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < zf_compact_pages_workspace_size(num_pages)) return ZF_ERR_WORKSPACE_TOO_SMALL;
  CompactArgs a{};
  a.page_table = page_table;
  a.pages_held = pages_held;
  a.out_table = new_page_table;
  a.free_pages = free_pages;
  a.free_pos = free_pos;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.used = static_cast<uint32_t*>(workspace);
  a.to = static_cast<int32_t*>(workspace) + (static_cast<size_t>(num_pages) + 31) / 32;
  a.status = status;
  a.batch = batch;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  const long long most = static_cast<long long>(batch) * max_pages;
  return launch_cluster(compact_kernel, 2, ctas_for(most > num_pages ? most : num_pages), static_cast<size_t>(batch) * 4,
                        ZF_MAX_BATCH * 4, static_cast<cudaStream_t>(stream), a);
}

extern "C" zf_status zf_q4_copy_pages(const zf_q4_cache* c, const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
  const zf_status st = check_q4_cache(c);
  if (st != ZF_OK) return st;
  if (n < 0) return ZF_ERR_INVALID_ARGUMENT;
  if (n == 0) return ZF_OK;
  if (!words_ok({src, dst})) return ZF_ERR_INVALID_ARGUMENT;
  CopyArgs a{};
  a.records = c->records;
  a.src = src;
  a.dst = dst;
  a.status = c->status;
  a.page_bytes = static_cast<size_t>(c->num_kv_heads) * (c->page_size / ZF_BLOCK_TOKENS) * kQ4Record;
  a.n = n;
  a.num_pages = c->num_pages;
  const long long chunks = static_cast<long long>((a.page_bytes + kCopyBytes - 1) / kCopyBytes);
  if (chunks > INT_MAX) return ZF_ERR_UNSUPPORTED;
  a.chunks = static_cast<int32_t>(chunks);
  const long long items = static_cast<long long>(n) * a.chunks;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items < 1216 ? items : 1216));       // 152 SMs x 8 resident CTAs
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, copy_kernel, a) == cudaSuccess ? ZF_OK : ZF_ERR_CUDA;
}
