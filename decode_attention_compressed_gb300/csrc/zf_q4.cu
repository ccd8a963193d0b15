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
// One thread owns one block of K and the same block of V: it reads 32 contiguous bytes of each, needs
// no exchange with other lanes and writes 8 code bytes and one scale byte of each; 8 consecutive
// threads cover the 64-byte code rows of a token and kv head.
#include <cuda_runtime.h>
#include <stdint.h>

#include "zf_q4.cuh"

namespace zf {

constexpr int kQ4Threads = 128;

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

// Thread index -> (entry, head, block): [n][hkv][8].
struct Q4Place {
  uint8_t* rec;
  size_t src;               // first value of the block in a [n][hkv][128] array
  int tok, block;
  bool in;                  // within the call
};
__device__ __forceinline__ Q4Place q4_place(const Q4Args& a) {
  const size_t g = static_cast<size_t>(blockIdx.x) * kQ4Threads + threadIdx.x;
  const uint32_t row = static_cast<uint32_t>(g >> 3);           // entry * hkv + head, below 2^31
  Q4Place p;
  p.block = static_cast<int>(g & 7);
  p.src = g * 16;
  p.tok = 0;
  p.in = (g >> 3) < static_cast<size_t>(a.n) * a.hkv;
  p.rec = nullptr;
  if (p.in) {
    const int i = static_cast<int>(row / static_cast<uint32_t>(a.hkv));
    const int h = static_cast<int>(row - static_cast<uint32_t>(i) * a.hkv);
    p.rec = q4_record(a, i, h, p.tok, h == 0 && p.block == 0);
  }
  return p;
}

// One block of 16 BF16 values (as eight words) -> codes and scale byte; odd: a NaN or an infinity among
// them.  The largest magnitude is found on the bit patterns, two at a time; a block with something that is
// not finite, or beyond every code, is cleaned up first.
__device__ __forceinline__ uint2 q4_quantise(const uint32_t (&w)[8], float inv, uint32_t& sbyte, bool& odd) {
  float t[16];
  uint32_t big2 = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    big2 = __vmaxu2(big2, w[j] & 0x7FFF7FFFu);
    t[2 * j] = bf16lo_to_f32(w[j]) * inv;
    t[2 * j + 1] = bf16hi_to_f32(w[j]) * inv;
  }
  const uint32_t big = max(big2 & 0xFFFFu, big2 >> 16);
  float amax = __uint_as_float(big << 16) * inv;      // rounding keeps the order: this is max |t|
  if (!(amax <= 65536.f)) {                           // 6 * 448 and less are the values that codes reach
    odd |= big >= 0x7F80u;
    amax = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      t[j] = t[j] != t[j] ? 0.f : fminf(fmaxf(t[j], -65536.f), 65536.f);       // saturates either way
      amax = fmaxf(amax, fabsf(t[j]));
    }
  }
  // scale: e4m3 of max / 6, at least its smallest positive number
  uint16_t pair;
  const float want = amax > 0.f ? fmaxf(__fdiv_rn(amax, 6.f), 0.001953125f) : 0.f;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(0.f), "f"(want));
  sbyte = pair & 0xFFu;
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
  return make_uint2(codes[0], codes[1]);
}

__global__ void __launch_bounds__(kQ4Threads) q4_write_kernel(const Q4Args a) {
  allow_next_grid();
  wait_prior_grid();
  const Q4Place p = q4_place(a);
  if (!p.rec) return;
  uint32_t w[2][8];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const uint4* src = reinterpret_cast<const uint4*>((v ? a.v : a.k) + p.src);
    const uint4 lo = src[0], hi = src[1];
    w[v][0] = lo.x; w[v][1] = lo.y; w[v][2] = lo.z; w[v][3] = lo.w;
    w[v][4] = hi.x; w[v][5] = hi.y; w[v][6] = hi.z; w[v][7] = hi.w;
  }
  bool odd = false;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    uint32_t sbyte;
    const uint2 codes = q4_quantise(w[v], v ? a.v_inv : a.k_inv, sbyte, odd);
    *reinterpret_cast<uint2*>(p.rec + (v ? q4_v_code_at(p.tok, p.block) : q4_k_code_at(p.tok, p.block))) = codes;
    p.rec[v ? q4_v_scale_at(p.tok, p.block) : q4_k_scale_at(p.tok, p.block)] = static_cast<uint8_t>(sbyte);
  }
  if (odd) report(a.status, ZF_DEV_NOT_FINITE);
}

// Values of the listed tokens as BF16: code * s * cache scale, rounded once (exact when the cache
// scale is a power of two).  Skipped and bad entries read as zeros.
__global__ void __launch_bounds__(kQ4Threads) q4_read_kernel(const Q4Args a) {
  allow_next_grid();
  wait_prior_grid();
  const Q4Place p = q4_place(a);
  if (!p.in) return;
  uint2 codes[2] = {};
  uint32_t sbyte[2] = {0u, 0u};
  if (p.rec) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      codes[v] = *reinterpret_cast<const uint2*>(p.rec + (v ? q4_v_code_at(p.tok, p.block) : q4_k_code_at(p.tok, p.block)));
      sbyte[v] = p.rec[v ? q4_v_scale_at(p.tok, p.block) : q4_k_scale_at(p.tok, p.block)] & 0x7Fu;
    }
  }
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    // code * s is exact in float (two and four significant bits)
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(sbyte[v] << 7))) * kQ4ScaleFactor;
    const float g_scale = v ? a.v_scale : a.k_scale;
    uint32_t out[8];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t h[4];
      q4_decode4(half ? codes[v].y : codes[v].x, h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        out[4 * half + j] = pack_bf16x2(c.x * s * g_scale, c.y * s * g_scale);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>((v ? a.v_out : a.k_out) + p.src);
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
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
  const long long rows = static_cast<long long>(n) * c->num_kv_heads;
  if (rows > 0x7FFFFFFFll) return ZF_ERR_UNSUPPORTED;
  const long long blocks = (rows * 8 + kQ4Threads - 1) / kQ4Threads;
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
