// Decode attention over the 8-bit KV cache: peagle_decode_attention_quant.
//
// The draft block's attention ("P-EAGLE: A Technical Deep Dive into Parallel Speculative
// Decoding", section "2. The P-EAGLE Parallel Drafter": the K rows of a request attend over
// the cache and the rows before them), reading codes and block scales.
#include <math.h>

#include "kv_quant.cuh"

namespace peagle {
namespace kvq {

struct AttnQuantArgs {
  const uint8_t* k;        // this layer's codes [batch slots][nkv][capacity][hd]
  const uint8_t* v;
  const float* k_scale;    // [batch slots][nkv][capacity / block]
  const float* v_scale;
  const void* q;
  int64_t q_stride;
  void* out;
  float* lse;
  const int* seq_lens;
  int* errors;
  float* work;
  int batch, K, nq, nkv, capacity, block_shift, causal, window;
  float scale;
};

// The slots [begin, end) that row j of a request of length len sees; empty when end <= begin.
__device__ __forceinline__ void row_span(const AttnQuantArgs& a, int len, int j, int& begin,
                                         int& end) {
  end = a.causal ? len + j + 1 : len;
  begin = a.window > 0 ? max(0, len + j - a.window + 1) : 0;
}

__device__ __forceinline__ bool request_fits(const AttnQuantArgs& a, int len) {
  return len >= 0 && len <= a.capacity - (a.causal ? a.K : 0);
}

// One warp per (request, draft row, query head); each lane keeps the running maximum, sum and
// output of every 32nd slot.
template <int HD, typename T>
__global__ void __launch_bounds__(128) attn_quant_simple_kernel(AttnQuantArgs a) {
  pdl_enter();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int item = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= a.K * a.nq) return;
  const int j = item / a.nq, h = item % a.nq, g = h / (a.nq / a.nkv);
  const int len = a.seq_lens[b];
  if (!request_fits(a, len)) {
    if (item == 0 && lane == 0) raise_error(a.errors, PEAGLE_DEV_KV_OVERFLOW);
    return;
  }
  int begin, end;
  row_span(a, len, j, begin, end);
  const int64_t unit = (int64_t)b * a.nkv + g;
  const int64_t row = (int64_t)b * a.K + j;
  const T* q = (const T*)a.q + row * a.q_stride + (int64_t)h * HD;
  float m = -INFINITY, sum = 0.f, o[HD];
#pragma unroll
  for (int d = 0; d < HD; ++d) o[d] = 0.f;
  for (int t = begin + lane; t < end; t += 32) {
    const uint8_t* k = a.k + (unit * a.capacity + t) * HD;
    const uint8_t* v = a.v + (unit * a.capacity + t) * HD;
    const int64_t at = unit * (a.capacity >> a.block_shift) + (t >> a.block_shift);
    float x = 0.f;
    for (int d = 0; d < HD; d += 2) {
      const float2 f = cvt_e4m3x2_f32x2(*(const uint16_t*)(k + d));
      x += ld(q + d) * f.x + ld(q + d + 1) * f.y;
    }
    x *= a.k_scale[at] * a.scale;
    const float top = fmaxf(m, x);
    const float keep = m == -INFINITY ? 0.f : expf(m - top), p = expf(x - top);
    m = top;
    sum = sum * keep + p;
    const float w = p * a.v_scale[at];
    for (int d = 0; d < HD; d += 2) {
      const float2 f = cvt_e4m3x2_f32x2(*(const uint16_t*)(v + d));
      o[d] = o[d] * keep + w * f.x;
      o[d + 1] = o[d + 1] * keep + w * f.y;
    }
  }
  const float top = warp_max(m);
  const float f = m == -INFINITY ? 0.f : expf(m - top);
  const float total = warp_sum(sum * f);
  T* out = (T*)a.out + (row * a.nq + h) * HD;
#pragma unroll
  for (int d = 0; d < HD; ++d) {
    const float x = warp_sum(o[d] * f);
    if (lane == (d & 31)) st(out + d, end > begin ? x / total : 0.f);
  }
  if (a.lse && lane == 0) a.lse[row * a.nq + h] = end > begin ? top + logf(total) : -INFINITY;
}

}  // namespace kvq
}  // namespace peagle

using namespace peagle;
using namespace peagle::kvq;

static int check_attention(const peagle_kv_quant* kv, int32_t batch, int32_t K,
                           int32_t n_q_heads) {
  const int rc = check_cache(kv, 0, batch);
  if (rc != PEAGLE_OK) return rc;
  if (K < 1 || n_q_heads < 1 || n_q_heads % kv->n_kv_heads) return PEAGLE_ERR_INVALID;
  if (K > 128 || K * (int64_t)(n_q_heads / kv->n_kv_heads) > 128) return PEAGLE_ERR_UNSUPPORTED;
  return PEAGLE_OK;
}

extern "C" int64_t peagle_decode_attention_quant_workspace(const peagle_kv_quant* kv,
                                                           int32_t batch, int32_t K,
                                                           int32_t n_q_heads) {
  const int rc = check_attention(kv, batch, K, n_q_heads);
  if (rc != PEAGLE_OK) return rc;
  return 256;
}

extern "C" int peagle_decode_attention_quant(const peagle_kv_quant* kv, int32_t layer,
                                             int32_t batch, int32_t K, int32_t n_q_heads,
                                             const void* q, int32_t dtype, int64_t q_stride,
                                             const int32_t* seq_lens, int32_t causal,
                                             int32_t window, float scale, void* out,
                                             float* out_lse, void* workspace,
                                             int64_t workspace_bytes, void* stream) {
  const int64_t need = peagle_decode_attention_quant_workspace(kv, batch, K, n_q_heads);
  if (need < 0) return (int)need;
  if (layer < 0 || layer >= kv->n_layers || !q || !seq_lens || !out || !workspace ||
      (causal != 0 && causal != 1) || window < 0 || !isfinite(scale))
    return PEAGLE_ERR_INVALID;
  if (dtype != PEAGLE_F32 && dtype != PEAGLE_BF16) return PEAGLE_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) || !aligned(out_lse, 4) ||
      q_stride % (dtype == PEAGLE_F32 ? 4 : 8))
    return PEAGLE_ERR_INVALID;
  if (workspace_bytes < need) return PEAGLE_ERR_CAPACITY;
  const int64_t unit = (int64_t)layer * kv->batch * kv->n_kv_heads;
  AttnQuantArgs a;
  a.k = (const uint8_t*)kv->k + unit * kv->capacity * kv->head_dim;
  a.v = (const uint8_t*)kv->v + unit * kv->capacity * kv->head_dim;
  a.k_scale = kv->k_scale + unit * (kv->capacity / kv->block);
  a.v_scale = kv->v_scale + unit * (kv->capacity / kv->block);
  a.q = q;
  a.q_stride = q_stride ? q_stride : (int64_t)n_q_heads * kv->head_dim;
  a.out = out, a.lse = out_lse, a.seq_lens = seq_lens, a.errors = kv->errors;
  a.work = (float*)workspace;
  a.batch = batch, a.K = K, a.nq = n_q_heads, a.nkv = kv->n_kv_heads, a.capacity = kv->capacity;
  a.block_shift = kv->block == 16 ? 4 : kv->block == 32 ? 5 : kv->block == 64 ? 6 : 7;
  a.causal = causal, a.window = window, a.scale = scale;
  const dim3 grid((unsigned)cdiv(K * n_q_heads, 4), (unsigned)batch);
  auto launch = [&](void (*kernel)(AttnQuantArgs)) {
    return launch_pdl(kernel, grid, dim3(128), 0, (cudaStream_t)stream, a);
  };
  const bool f32 = dtype == PEAGLE_F32;
  const cudaError_t e =
      kv->head_dim == 64
          ? launch(f32 ? attn_quant_simple_kernel<64, float> : attn_quant_simple_kernel<64, bf16>)
          : launch(f32 ? attn_quant_simple_kernel<128, float> : attn_quant_simple_kernel<128, bf16>);
  return e == cudaSuccess ? PEAGLE_OK : PEAGLE_ERR_CUDA;
}
