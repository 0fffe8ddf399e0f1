// The 8-bit KV cache (peagle_kv_quant): argument checks and the e4m3 conversions that its
// kernels share (kv_quant.cu writes and reads the cache, kv_quant_attn.cu attends over it).
//
// The kernels start before the one ahead of them in the stream has ended (programmatic launch), so
// nothing they read is constant over their lifetime: plain loads, none through the read-only path.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace peagle {
namespace kvq {

// Two e4m3 codes (low byte first) as f16: exact, every e4m3 value is an f16 value.
__device__ __forceinline__ uint32_t cvt_e4m3x2_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// Four codes: the low two and the high two.
__device__ __forceinline__ void cvt_e4m3x4_f16x2(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ float2 cvt_e4m3x2_f32x2(uint16_t c) {
  const uint32_t h = cvt_e4m3x2_f16x2(c);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Two fp32 values as e4m3 codes, `lo` in the low byte: round to nearest even, NaN to NaN.
__device__ __forceinline__ uint16_t cvt_f32x2_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// NaN codes of a word: 0x80 in each such byte.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

__device__ __forceinline__ void raise_error(int* err, unsigned bits) {
  if (err) atomicOr((unsigned*)err, bits);
}

static inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p % to) == 0; }

// What every call checks of the cache, the layer and the batch.
static inline int check_cache(const peagle_kv_quant* kv, int32_t layer, int32_t batch) {
  if (!kv || !kv->k || !kv->v || !kv->k_scale || !kv->v_scale) return PEAGLE_ERR_INVALID;
  if (kv->n_layers < 1 || kv->n_layers > 65535 || kv->batch < 1 || kv->batch > 65535 ||
      kv->n_kv_heads < 1 || kv->n_kv_heads > 65535 || kv->capacity < 1)
    return PEAGLE_ERR_INVALID;
  if (kv->head_dim != 64 && kv->head_dim != 128) return PEAGLE_ERR_UNSUPPORTED;
  if (kv->block != 16 && kv->block != 32 && kv->block != 64 && kv->block != 128)
    return PEAGLE_ERR_UNSUPPORTED;
  // (slots above 2^30 would leave no room for the position arithmetic in 32 bits)
  if (kv->capacity % kv->block || kv->capacity > (1 << 30)) return PEAGLE_ERR_INVALID;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->k_scale, 4) ||
      !aligned(kv->v_scale, 4) || !aligned(kv->errors, 4))
    return PEAGLE_ERR_INVALID;
  if (layer < -1 || layer >= kv->n_layers || batch < 1) return PEAGLE_ERR_INVALID;
  if (batch > kv->batch) return PEAGLE_ERR_CAPACITY;
  return PEAGLE_OK;
}

}  // namespace kvq
}  // namespace peagle
