// What the two decode attention kernels over the 8-bit cache share (kv_quant_attn.cu on warps'
// products, kv_quant_attn_tc.cu on tcgen05): arguments, which slots a row sees, the equal shares of
// the call's tiles, and the result of a row.
#pragma once

#include <math.h>

#include <type_traits>

#include "kv_quant.cuh"
#include "tc_ptx.cuh"

namespace peagle {
namespace kvq {

constexpr int CTAS = 152;      // GB300's SMs
constexpr int MAX_ROWS = 128;  // query rows a kv head
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float NO_REF = -3.0e38f;  // the reference of a row that has seen no slot

// A reference puts the largest weight at 2^SHIFT, and it may grow to 2^LIM before the reference moves
// (f16 ends at 2^16).  Below 2^-14 weights lose bits of their 11 and below 2^-25 all of them, while
// the sum of weights keeps them: n slots lose at most n 2^-(25 + SHIFT) of the largest weight, 2^-14
// for bf16 queries over 131072 slots.  Where one slot outweighs a long flat tail, that is the tail's
// share: a SHIFT of -4 (room for growth of 2^19) took 1 .. 8 % less time, but one slot 15 nats above
// 32768 others of 256 times its value came out 72 % too small.  The price of 2^9 of room is that
// references move more often: 64 requests of 300 .. 4100 slots with 64 query rows (tcgen05) 109.2 us
// in a graph for 100.9, 16 of 1024 .. 8192 with 20 rows 53.1 for 51.2, long contexts the same.  (2^10:
// 114.1 and 55.3; 2^13: 118.2 and 57.6.)  The second part of an fp32 weight needs the range below its
// first, so there the largest is put at 2^13.
constexpr float SHIFT_BF16 = 6.f, SHIFT_F32 = 13.f, LIM = 15.f;

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
  int split;               // > 0: a cluster of that many CTAs (a power of two) takes whole heads,
                           // and there is no second step
  float scale;             // of the scores, with log2(e)
  unsigned long long wait_ns;  // bound of the tcgen05 kernel's waits
  int stall;               // the Wait whose barriers want one arrival more than come, or -1
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
// 1 / c of a value scale from 2^-124 to the largest float (rcp alone gives 0 for subnormal results;
// below, where sums of w / c leave fp32 in any case, 2^124 stands for it).
__device__ __forceinline__ float inverse_scale(float c) {
  return rcp(fmaxf(c, 0x1p-124f) * 0.25f) * 0.25f;
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
// query rows of one), which costs `entry` tiles besides its own.
template <int TILE>
struct Segment {
  int b, h, len;
  int first_tile, tiles, entry;
  int at;  // of its first tile, relative to the CTA's share (negative: it began before)
  // The next one; false when it is not in the share of n any more.
  __device__ __forceinline__ bool next(const AttnQuantArgs& a, int n) {
    at += tiles + entry;
    if (at >= n) return false;
    if (++h < a.heads) return true;
    h = 0;
    do {
      if (++b >= a.batch) return false;
      len = a.seq_lens[b];
      tiles = request_tiles<TILE>(a, len, first_tile);
    } while (!tiles);
    cut(a);
    return true;
  }
  // Of a request's tiles those of this CTA of its cluster, none perhaps.
  __device__ __forceinline__ void cut(const AttnQuantArgs& a) {
    if (a.split < 2) return;
    const int shift = __ffs(a.split) - 1, r = (int)tc::cluster_ctarank(), from = tiles * r >> shift;
    tiles = (tiles * (r + 1) >> shift) - from;
    first_tile += from;
  }
};

// This CTA's share of the call: `seg`, where it begins, its cost n, where it lies (lo) and how long
// every share is.  False when it holds no tile.  A head's entry (its queries, the first tile's
// references, the join of the streams) counts as up to ENTRY tiles.  Where a CTA has fewer tiles
// than that, it counts as a share: then no CTA has to enter two heads, and no more CTAs than heads
// stay idle.  Every warp finds the share for itself, a lane summing up consecutive requests, so
// nothing waits on a barrier.  (The host has checked that all fits 31 bits.)
template <int TILE, int ENTRY>
__device__ __forceinline__ bool find_share(const AttnQuantArgs& a, int least, Segment<TILE>& seg,
                                           int& n, int& lo, int& share) {
  const int lane = threadIdx.x & 31, per = (a.batch + 31) / 32;
  const int b0 = min(lane * per, a.batch), b1 = min(b0 + per, a.batch);
  int my_tiles = 0, my_requests = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int len = a.seq_lens[b];
    int first;
    const int tiles = request_tiles<TILE>(a, len, first);
    my_tiles += tiles;
    my_requests += tiles > 0;
    if (blockIdx.x == 0 && threadIdx.x < 32 && !request_fits(a, len))
      raise_error(a.errors, PEAGLE_DEV_KV_OVERFLOW);
  }
  const int all_tiles = __reduce_add_sync(0xffffffffu, my_tiles) * a.heads;
  seg.entry = min(ENTRY, all_tiles / CTAS + 1);
  const int mine = (my_tiles + my_requests * seg.entry) * a.heads;
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  const int total = __shfl_sync(0xffffffffu, upto, 31);
  share = max(least, (total + CTAS - 1) / CTAS);
  lo = share * blockIdx.x;
  n = min(share, total - lo);
  if (n <= 0) return false;
  const int who = __ffs(__ballot_sync(0xffffffffu, lo >= upto - mine && lo < upto)) - 1;
  int before = __shfl_sync(0xffffffffu, upto - mine, who);
  int cost;
  seg.b = __shfl_sync(0xffffffffu, b0, who) - 1;
  do {
    seg.len = a.seq_lens[++seg.b];
    seg.tiles = request_tiles<TILE>(a, seg.len, seg.first_tile);
    cost = seg.tiles ? (seg.tiles + seg.entry) * a.heads : 0;
    before += cost;
  } while (lo >= before);
  const int in = lo - (before - cost);
  seg.h = in / (seg.tiles + seg.entry);
  seg.at = seg.entry - (in - seg.h * (seg.tiles + seg.entry));
  return seg.at < n;
}

// The rows of heads [h, h + heads) of a request none of whose rows sees a slot: zeros and -inf.
template <int HD, typename T>
__device__ __forceinline__ void write_empty(const AttnQuantArgs& a, int req, int h, int heads) {
  const int nq = a.nkv * a.G, n = heads * a.G;
  for (int j = 0; j < a.K; ++j) {
    const int64_t row = ((int64_t)req * a.K + j) * nq + h * a.G;
    for (int i = threadIdx.x; i < n * HD; i += blockDim.x) st((T*)a.out + row * HD + i, 0.f);
    if (a.lse)
      for (int i = threadIdx.x; i < n; i += blockDim.x) a.lse[row + i] = -INFINITY;
  }
}

// find_share for a call in one step: equal numbers of consecutive heads a cluster, and of each head
// this CTA's part.  Writes the heads that see no slot.
template <int HD, typename T, int TILE>
__device__ __forceinline__ bool find_heads(const AttnQuantArgs& a, Segment<TILE>& seg, int& n) {
  const int shift = __ffs(a.split) - 1;
  const int clusters = gridDim.x >> shift, all = a.batch * a.heads;
  const int per = (all + clusters - 1) / clusters;
  const int begin = min(per * (int)(blockIdx.x >> shift), all), end = min(begin + per, all);
  const bool lead = a.split == 1 || (int)tc::cluster_ctarank() == 0;
  n = 0;
  seg.entry = 1, seg.at = 0;  // (the entry comes after the tiles here: a head without any counts too)
  for (int b = begin / a.heads; b * a.heads < end; ++b) {
    const int h = max(begin - b * a.heads, 0), heads = min(end - b * a.heads, a.heads) - h;
    Segment<TILE> x = seg;
    x.b = b, x.h = h, x.len = a.seq_lens[b];
    x.tiles = request_tiles<TILE>(a, x.len, x.first_tile);
    if (!request_fits(a, x.len)) {
      if (lead && threadIdx.x == 0) raise_error(a.errors, PEAGLE_DEV_KV_OVERFLOW);
    } else if (!x.tiles) {
      if (lead) write_empty<HD, T>(a, b, h, heads);
    } else {
      x.cut(a);
      if (!n) seg = x;
      n += heads * (x.tiles + seg.entry);
    }
  }
  return n > 0;
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
  if (l == INFINITY) l = NAN;  // (value scales so small that the sum of w / c left fp32)
  inv = none ? 0.f : rcp(l);
  const int64_t to = (int64_t)req * a.K * (a.nkv * a.G) + at;
  if (first && a.lse) a.lse[to] = none ? -INFINITY : (m + lg2(l)) * LN2;
  return (T*)a.out + to * hd;
}

// The kernels' second step (kv_quant_attn.cu): joins the pieces of heads that several CTAs worked
// on.  rowmajor: how the pieces' outputs lie in the workspace.
cudaError_t launch_join(int hd, bool f32, bool rowmajor, const AttnQuantArgs& a, int ntiles,
                        cudaStream_t s);
// The tcgen05 kernel, the calls it takes, and the rows of its workspace slots (kv_quant_attn_tc.cu).
bool attn_quant_tc_takes(int hd, bool f32, int rows, int64_t slots);
int attn_quant_tc_rows(int rows);
cudaError_t launch_attention_tc(int hd, int rows, AttnQuantArgs a, cudaStream_t s);

}  // namespace kvq
}  // namespace peagle
