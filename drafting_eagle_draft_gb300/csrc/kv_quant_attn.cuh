// What the two decode attention kernels over the 8-bit cache share (kv_quant_attn.cu on warps'
// products, kv_quant_attn_tc.cu on tcgen05): arguments, which slots a row sees, the equal shares of
// the call's tiles, and the result of a row.
#pragma once

#include <math.h>

#include <type_traits>

#include "kv_quant.cuh"

namespace peagle {
namespace kvq {

constexpr int CTAS = 152;      // GB300's SMs
constexpr int MAX_ROWS = 128;  // query rows a kv head
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float NO_REF = -3.0e38f;  // the reference of a row that has seen no slot

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
  int4* desc;              // [CTAS]: request, head, last CTA of the piece chain (or -1)
  float* work;             // [CTAS][2] slots of partial results
  int batch, K, G, nkv, capacity, block_shift, causal, window;
  int heads;               // work items a request: kv heads x parts of their query rows
  int groups;              // warps that share a stream's tiles, each NT x 8 query rows
  int stages;
  int part_rows;           // query rows of a part
  float scale;             // of the scores, with log2(e)
};

// Slots [begin, end) that row j of a request of length len sees; empty when end <= begin.
__device__ __forceinline__ int row_begin(const AttnQuantArgs& a, int len, int j) {
  return a.window > 0 ? max(0, len + j - a.window + 1) : 0;
}
__device__ __forceinline__ int row_end(const AttnQuantArgs& a, int len, int j) {
  return a.causal ? len + j + 1 : len;
}
__device__ __forceinline__ bool request_fits(const AttnQuantArgs& a, int len) {
  return len >= 0 && len <= a.capacity - (a.causal ? a.K : 0);
}
// Tiles of TILE slots, [first, first + count), that some row of a request sees.
template <int TILE>
__device__ __forceinline__ int request_tiles(const AttnQuantArgs& a, int len, int& first) {
  first = 0;
  if (!request_fits(a, len)) return 0;
  const int lo = row_begin(a, len, 0), hi = row_end(a, len, a.K - 1);
  if (hi <= lo) return 0;
  first = lo / TILE;
  return (hi + TILE - 1) / TILE - first;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Where a CTA's walk over the tiles stands: one head of a request (a kv head, or a part of the
// query rows of one), which costs ENTRY tiles besides its own.
template <int TILE, int ENTRY>
struct Segment {
  int b, h, len;
  int first_tile, tiles;
  int at;  // of its first tile, relative to the CTA's share (negative: it began before)
  // The next one; false when it is not in the share of n any more.
  __device__ __forceinline__ bool next(const AttnQuantArgs& a, int n) {
    at += tiles + ENTRY;
    if (at >= n) return false;
    if (++h < a.heads) return true;
    h = 0;
    do {
      if (++b >= a.batch) return false;
      len = a.seq_lens[b];
      tiles = request_tiles<TILE>(a, len, first_tile);
    } while (!tiles);
    return true;
  }
};

// Sum over the W warps' threads of v before this one, and over all of them.
template <int W>
__device__ __forceinline__ long long block_scan(long long v, long long* red, long long& total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) red[wid] = x;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const long long s = red[i];
    if (i < wid) before += s;
    total += s;
  }
  return before + x - v;
}


// This CTA's share of the call: `seg`, where it begins, its cost n, where it lies (lo) and how long
// every share is.  False when it holds no tile.  All W x 32 threads.
template <int W, int TILE, int ENTRY>
__device__ __forceinline__ bool find_share(const AttnQuantArgs& a, int least, Segment<TILE, ENTRY>& seg,
                                           int& n, long long& lo, long long& share) {
  __shared__ long long red[W];
  __shared__ long long found;
  __shared__ int found_b;
  long long total = 0, cost = 0, before = 0;
  int first;
  auto cost_of = [&](int b) {
    const int tiles = b < a.batch ? request_tiles<TILE>(a, a.seq_lens[b], first) : 0;
    return tiles ? (long long)(tiles + ENTRY) * a.heads : 0;
  };
  for (int b0 = 0; b0 < a.batch; b0 += W * 32) {
    const int b = b0 + threadIdx.x;
    cost = cost_of(b);
    if (blockIdx.x == 0 && b < a.batch && !request_fits(a, a.seq_lens[b]))
      raise_error(a.errors, PEAGLE_DEV_KV_OVERFLOW);
    long long part;
    before = block_scan<W>(cost, red, part);
    total += part;
  }
  share = (total + CTAS - 1) / CTAS;
  share = share < least ? least : share;
  lo = share * blockIdx.x;
  n = (int)(total - lo < share ? total - lo : share);
  long long base = 0;
  for (int b0 = 0; b0 < a.batch && lo < total; b0 += W * 32) {
    if (a.batch > W * 32) {
      cost = cost_of(b0 + threadIdx.x);
      long long part;
      before = base + block_scan<W>(cost, red, part);
      base += part;
    }
    if (cost && lo >= before && lo < before + cost) {
      found = before;
      found_b = b0 + threadIdx.x;
    }
  }
  __syncthreads();
  if (lo >= total) return false;
  seg.b = found_b;
  seg.len = a.seq_lens[seg.b];
  seg.tiles = request_tiles<TILE>(a, seg.len, seg.first_tile);
  const long long in = lo - found;
  seg.h = (int)(in / (seg.tiles + ENTRY));
  seg.at = ENTRY - (int)(in % (seg.tiles + ENTRY));
  return seg.at < n;
}

// Two values of a row at consecutive head dims.
__device__ __forceinline__ void store2(float* p, float x, float y) {
  *reinterpret_cast<float2*>(p) = make_float2(x, y);
}
__device__ __forceinline__ void store2(bf16* p, float x, float y) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
}

// A row's result: its address in out and 1 / l (0 for a row that has seen nothing); writes its lse
// when `first`.  at: the row's place among its request's rows and heads.
template <typename T>
__device__ __forceinline__ T* finish_row(const AttnQuantArgs& a, int hd, int req, int at, float m,
                                         float l, bool first, float& inv) {
  const bool none = m == NO_REF && l == 0.f;  // (a row of NaN scores has no reference either)
  inv = none ? 0.f : 1.f / l;
  const int64_t to = (int64_t)req * a.K * (a.nkv * a.G) + at;
  if (first && a.lse) a.lse[to] = none ? -INFINITY : (m + log2f(l)) * LN2;
  return (T*)a.out + to * hd;
}

// The kernels' second step (kv_quant_attn.cu): joins the pieces of heads that several CTAs worked
// on.  rowmajor: how the pieces' outputs lie in the workspace.
cudaError_t launch_join(int hd, bool f32, bool rowmajor, const AttnQuantArgs& a, int ntiles,
                        cudaStream_t s);
// tcgen05 kernel, its shapes, and the workspace slot's rows (kv_quant_attn_tc.cu).
bool attn_quant_tc_takes(int hd, bool f32, int rows, int64_t slots);
int attn_quant_tc_rows(int rows);
cudaError_t launch_attention_tc(int hd, int rows, AttnQuantArgs a, cudaStream_t s);

}  // namespace kvq
}  // namespace peagle
