// The 4-bit cache record shared by the zf_q4_* kernels (layout and number formats: include/zf.h).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "zf_device.cuh"
#include "zf_host.h"

namespace zf {

constexpr int kQ4Record = ZF_Q4_RECORD_BYTES;      // 16 tokens of one (page, kv head), K and V
constexpr int kQ4VCodes = 1024, kQ4KScales = 2048, kQ4VScales = 2176;
static_assert(kQ4VScales + 128 == kQ4Record, "record layout");
// Scales are decoded as (byte & 0x7f) << 7, the bits of a half: exponent and fraction fields of
// e4m3 land in those of fp16, subnormals included, and the value comes out 2^-8 of the scale.
// (No byte decodes to a NaN: 0x7f, which the writer never stores, reads as 480.)
constexpr float kQ4ScaleFactor = 256.f;

// Byte offsets within a record.
__host__ __device__ constexpr int q4_k_code_at(int tok, int block) { return tok * 64 + block * 8; }
__host__ __device__ constexpr int q4_v_code_at(int tok, int block) {
  return kQ4VCodes + tok * 64 + ((block ^ ((tok & 2) << 1)) * 8);
}
__host__ __device__ constexpr int q4_k_scale_at(int tok, int block) {
  return kQ4KScales + (tok & 7) * 16 + (block >> 1) * 4 + (tok >> 3) * 2 + (block & 1);
}
__host__ __device__ constexpr int q4_v_scale_at(int tok, int block) {
  return kQ4VScales + block * 16 + ((tok & 7) >> 1) * 4 + (tok >> 3) * 2 + (tok & 1);
}

// Four bytes of two e2m1 codes each -> four half pairs (low nibble in the low half).
__device__ __forceinline__ void q4_decode4(uint32_t bytes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(bytes));
}

// Eight floats -> e2m1 codes, nearest even, saturating at 6 (float j in nibble j).
__device__ __forceinline__ uint32_t q4_encode8(const float (&q)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Argument checks of a 4-bit cache descriptor.
inline zf_status check_q4_cache(const zf_q4_cache* c) {
  if (!c) return ZF_ERR_INVALID_ARGUMENT;
  if (c->head_dim != ZF_HEAD_DIM) return ZF_ERR_INVALID_ARGUMENT;
  if (c->page_size < ZF_BLOCK_TOKENS || c->page_size % ZF_BLOCK_TOKENS != 0) return ZF_ERR_INVALID_ARGUMENT;
  if (c->page_size > ZF_MAX_PAGE_SIZE) return ZF_ERR_UNSUPPORTED;
  if (c->num_kv_heads < 1 || c->num_pages < 0) return ZF_ERR_INVALID_ARGUMENT;
  if (c->num_pages > 0 && (!c->records || !aligned16(c->records))) return ZF_ERR_INVALID_ARGUMENT;
  // positive, and far enough from the ends of float for their reciprocals and the stored values
  for (const float s : {c->k_scale, c->v_scale})
    if (!(s >= 1e-30f && s <= 1e30f)) return ZF_ERR_INVALID_ARGUMENT;
  if (c->status && (reinterpret_cast<uintptr_t>(c->status) & 3u)) return ZF_ERR_INVALID_ARGUMENT;
  return ZF_OK;
}

}  // namespace zf
