// zf_q4_write_tokens and zf_q4_read_tokens: tokens quantised into a paged 4-bit cache, and back.
//
// Mathematics, per block of 16 channels (include/zf.h): t = x / scale of the cache (as a product
// with the reciprocal), a = max |t|, s = e4m3(a / 6) kept in [2^-9, 448] (0 when a = 0), code =
// e2m1(t / s), both to nearest even.  The quotient is needed exactly rounded (a value on the
// border between two codes must fall the same way everywhere): q = t r with r = 1/s correctly
// rounded, then q + (t - q s) r in two fused operations, which is the correctly rounded t / s
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
//
// Bound: bytes (512 in, 144 out per token and kv head; a decode step's few tokens: launch latency).
// One thread owns one block of K or of V: it reads 32 contiguous bytes, needs no exchange with
// other lanes and writes 8 code bytes and one scale byte; 8 consecutive threads cover a 64-byte
// code row.
#include <cuda_runtime.h>
#include <stdint.h>

#include "zf_q4.cuh"

namespace zf {

constexpr int kQ4Threads = 256;

struct Q4Args {
  uint8_t* records;
  int32_t* status;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* k_out;
  uint16_t* v_out;
  const int32_t* page_ids;
  const int32_t* positions;
  int32_t n, hkv, num_pages, page_size;
  float k_scale, v_scale, k_inv, v_inv;
};

// Record and token index of entry i's token for head h; null when the entry is skipped (position
// -1) or bad (reported by the caller's first thread of the entry).
__device__ __forceinline__ uint8_t* q4_record(const Q4Args& a, int i, int h, int& tok, bool tell) {
  const int pid = a.page_ids[i], pos = a.positions[i];
  if (pos == -1) return nullptr;
  if (pid < 0 || pid >= a.num_pages || pos < 0 || pos >= a.page_size) {
    if (tell) report(a.status, (pid < 0 || pid >= a.num_pages) ? ZF_DEV_BAD_PAGE_ID : ZF_DEV_BAD_N_VALID);
    return nullptr;
  }
  tok = pos & 15;
  return a.records + ((static_cast<size_t>(pid) * a.hkv + h) * (a.page_size >> 4) + (pos >> 4)) * kQ4Record;
}

// Thread index -> (entry, head, K or V, block): [n][hkv][2][8].
__global__ void __launch_bounds__(kQ4Threads) q4_write_kernel(const Q4Args a) {
  allow_next_grid();
  wait_prior_grid();
  const long long g = static_cast<long long>(blockIdx.x) * kQ4Threads + threadIdx.x;
  const int block = static_cast<int>(g & 7);
  const bool is_v = (g >> 3) & 1;
  const long long row = g >> 4;                       // entry * hkv + head
  if (row >= static_cast<long long>(a.n) * a.hkv) return;
  const int i = static_cast<int>(row / a.hkv), h = static_cast<int>(row - static_cast<long long>(i) * a.hkv);
  int tok = 0;
  uint8_t* rec = q4_record(a, i, h, tok, h == 0 && (g & 15) == 0);
  if (!rec) return;
  const uint4* src = reinterpret_cast<const uint4*>((is_v ? a.v : a.k) + row * ZF_HEAD_DIM + block * 16);
  const uint4 lo = src[0], hi = src[1];
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  const float inv = is_v ? a.v_inv : a.k_inv;
  float t[16];
  float amax = 0.f;
  bool odd = false;                                   // a NaN or an infinity among the values
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t bits = (j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16;
    odd |= (bits & 0x7F800000u) == 0x7F800000u;
    float x = __uint_as_float(bits) * inv;
    x = x != x ? 0.f : x;
    t[j] = fminf(fmaxf(x, -65536.f), 65536.f);        // beyond 6 * 448: saturates either way
    amax = fmaxf(amax, fabsf(t[j]));
  }
  if (odd) report(a.status, ZF_DEV_NOT_FINITE);
  // scale: e4m3 of max / 6, at least its smallest positive number
  uint16_t pair;
  const float want = amax > 0.f ? fmaxf(__fdiv_rn(amax, 6.f), 0.001953125f) : 0.f;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(0.f), "f"(want));
  const uint32_t sbyte = pair & 0xFFu;
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(sbyte << 7))) * kQ4ScaleFactor;
  const float r = sbyte ? __frcp_rn(s) : 0.f;
  uint32_t codes[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = t[8 * half + j];
      const float q0 = __fmul_rn(x, r);
      q[j] = __fmaf_rn(__fmaf_rn(-q0, s, x), r, q0);
    }
    codes[half] = q4_encode8(q);
  }
  *reinterpret_cast<uint2*>(rec + (is_v ? q4_v_code_at(tok, block) : q4_k_code_at(tok, block))) =
      make_uint2(codes[0], codes[1]);
  rec[is_v ? q4_v_scale_at(tok, block) : q4_k_scale_at(tok, block)] = static_cast<uint8_t>(sbyte);
}

// Values of the listed tokens as BF16: code * s * cache scale, rounded once (exact when the cache
// scale is a power of two).  Skipped and bad entries read as zeros.
__global__ void __launch_bounds__(kQ4Threads) q4_read_kernel(const Q4Args a) {
  allow_next_grid();
  wait_prior_grid();
  const long long g = static_cast<long long>(blockIdx.x) * kQ4Threads + threadIdx.x;
  const int block = static_cast<int>(g & 7);
  const bool is_v = (g >> 3) & 1;
  const long long row = g >> 4;
  if (row >= static_cast<long long>(a.n) * a.hkv) return;
  const int i = static_cast<int>(row / a.hkv), h = static_cast<int>(row - static_cast<long long>(i) * a.hkv);
  int tok = 0;
  const uint8_t* rec = q4_record(a, i, h, tok, h == 0 && (g & 15) == 0);
  uint32_t out[8] = {};
  if (rec) {
    const uint2 codes = *reinterpret_cast<const uint2*>(rec + (is_v ? q4_v_code_at(tok, block) : q4_k_code_at(tok, block)));
    const uint32_t sbyte = rec[is_v ? q4_v_scale_at(tok, block) : q4_k_scale_at(tok, block)] & 0x7Fu;
    // code * s is exact in float (two and four significant bits)
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(sbyte << 7))) * kQ4ScaleFactor;
    const float g_scale = is_v ? a.v_scale : a.k_scale;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t p[4];
      q4_decode4(half ? codes.y : codes.x, p);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&p[j]));
        out[4 * half + j] = pack_bf16x2(c.x * s * g_scale, c.y * s * g_scale);
      }
    }
  }
  uint4* dst = reinterpret_cast<uint4*>((is_v ? a.v_out : a.k_out) + row * ZF_HEAD_DIM + block * 16);
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

static zf_status q4_tokens(const zf_q4_cache* c, const void* k, const void* v, const int32_t* page_ids,
                           const int32_t* positions, int32_t n, bool write, void* stream) {
  const zf_status st = check_q4_cache(c);
  if (st != ZF_OK) return st;
  if (n < 0) return ZF_ERR_INVALID_ARGUMENT;
  if (n == 0) return ZF_OK;
  if (!k || !v || !page_ids || !positions || !aligned16(k) || !aligned16(v) ||
      (reinterpret_cast<uintptr_t>(page_ids) & 3u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return ZF_ERR_INVALID_ARGUMENT;
  const long long threads = static_cast<long long>(n) * c->num_kv_heads * 16;
  const long long blocks = (threads + kQ4Threads - 1) / kQ4Threads;
  if (blocks > 0x7FFFFFFFll) return ZF_ERR_UNSUPPORTED;
  Q4Args a{};
  a.records = c->records;
  a.status = c->status;
  if (write) {
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
  } else {
    a.k_out = static_cast<uint16_t*>(const_cast<void*>(k));
    a.v_out = static_cast<uint16_t*>(const_cast<void*>(v));
  }
  a.page_ids = page_ids;
  a.positions = positions;
  a.n = n;
  a.hkv = c->num_kv_heads;
  a.num_pages = c->num_pages;
  a.page_size = c->page_size;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.k_inv = 1.0f / c->k_scale;
  a.v_inv = 1.0f / c->v_scale;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kQ4Threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, write ? q4_write_kernel : q4_read_kernel, a) == cudaSuccess ? ZF_OK : ZF_ERR_CUDA;
}

}  // namespace zf

using namespace zf;

extern "C" zf_status zf_q4_write_tokens(const zf_q4_cache* cache, const uint16_t* k_tok, const uint16_t* v_tok,
                                        const int32_t* page_ids, const int32_t* positions, int32_t n, void* stream) {
  return q4_tokens(cache, k_tok, v_tok, page_ids, positions, n, true, stream);
}

extern "C" zf_status zf_q4_read_tokens(const zf_q4_cache* cache, const int32_t* page_ids, const int32_t* positions,
                                       int32_t n, uint16_t* k_out, uint16_t* v_out, void* stream) {
  return q4_tokens(cache, k_out, v_out, page_ids, positions, n, false, stream);
}
