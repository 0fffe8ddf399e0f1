// Writing and reading the 8-bit KV cache: peagle_append_kv_quant, peagle_read_kv_quant, and the
// open block set aside and put back (peagle_save_kv_quant, peagle_restore_kv_quant).
//
// The cache commit is part of every speculative round ("P-EAGLE: A Technical Deep Dive into
// Parallel Speculative Decoding", section "Technical Architecture"); the 8-bit form with a
// scale per block of slots is this library's.
#include "kv_quant.cuh"

namespace peagle {
namespace kvq {

struct RowsArgs {
  char* k;
  char* v;
  int64_t layer, batch, token, head;  // strides in elements
};

struct CacheArgs {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int* errors;
  int batch, heads, capacity;
  int layer0;
};

// Row counts of a request and whether they fit; raises the error bits when `report`.
__device__ __forceinline__ bool rows_fit(int at, int64_t n, int n_max, int capacity,
                                         int* errors, bool report) {
  if (n < 0 || n > n_max) {
    if (report) raise_error(errors, PEAGLE_DEV_BAD_COMMIT);
    return false;
  }
  if (at < 0 || at > capacity - n) {
    if (report) raise_error(errors, PEAGLE_DEV_KV_OVERFLOW);
    return false;
  }
  return true;
}

// 16 consecutive elements of a slot, as they were loaded: rows (16-byte aligned by the host's
// checks) or, in u[0], codes.
template <typename T>
struct Piece {
  static constexpr int N = sizeof(T);  // 16-byte words
  uint4 u[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4 x = u[i / 4];
    return i % 4 == 0 ? x.x : i % 4 == 1 ? x.y : i % 4 == 2 ? x.z : x.w;
  }
  // The largest magnitude of the row elements as fp32 bits (infinities and NaN are above 0x7f800000).
  __device__ __forceinline__ unsigned row_top() const {
    unsigned top = 0;
    if (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, word(i) & 0x7fffffffu);
    } else {  // two elements at a time, as 16-bit integers
#pragma unroll
      for (int i = 0; i < 8; ++i) top = __vmaxu2(top, word(i) & 0x7fff7fffu);
      top = max(top & 0xffff0000u, top << 16);
    }
    return top;
  }
  // Row elements 2 i and 2 i + 1.
  __device__ __forceinline__ float2 row_pair(int i) const {
    if (sizeof(T) == 4) return make_float2(__uint_as_float(word(2 * i)), __uint_as_float(word(2 * i + 1)));
    return make_float2(__uint_as_float(word(i) << 16), __uint_as_float(word(i) & 0xffff0000u));
  }
  // The values of codes 2 i and 2 i + 1.
  __device__ __forceinline__ float2 code_pair(int i, float scale) const {
    const uint32_t w = word(i / 2);
    const float2 f = cvt_e4m3x2_f32x2((uint16_t)(i % 2 ? w >> 16 : w));
    return make_float2(f.x * scale, f.y * scale);
  }
};

__device__ __forceinline__ unsigned magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ unsigned finite(unsigned bits) { return bits < 0x7f800000u ? bits : 0u; }

// A CTA encodes U / 2 consecutive blocks of slots of one (layer, request, kv head), keys and
// values: U units.
//
//   s = 2^e, the smallest with amax <= 448 s over the block's live values (448 = 1.75 x 2^8, so
//   e = E - 8 for amax = 1.m x 2^E with 1.m <= 1.75, else E - 7);  code = round(x / s)
//
// Each thread holds 16 consecutive elements of one slot of every unit in registers, as loaded:
// one pass over the rows (two or four 16-byte loads a unit), one exchange of maxima over the
// CTA, one 16-byte store a unit.  Scaling by a power of two is exact, so the only rounding is the
// conversion to e4m3; the committed slots of the first block are read back (16 codes a thread)
// and stored again only if their scale changed.  Heads run fastest over the grid: the rows of one
// token lie side by side.
//
// Long rows are bound by memory: U = 4 units in flight a CTA and 64 registers a thread (1024 threads
// an SM) hide the chain length -> rows -> maximum -> codes.  Counts are on the device, so CTAs for the
// longest request find the others ended: with LOOP a CTA goes on to the blocks `stride` further on, and
// there are a quarter as many.  Four prompts of 1001 .. 8192 bf16 tokens in 4 layers of 8 heads of 128:
// 78.8 us, 5.7 TB/s of the bytes they cannot do without (84 % of the measured copy rate), 85 without
// LOOP; 16 such prompts 290 (92 %) and 343, four in fp32 114 (97 %) and 134.  (Before LOOP: 99 with
// U = 2, 103 with 3 CTAs an SM.)  A draft block is bound by latency, and U = 2 spreads its units over
// more CTAs.  A few rows of many requests are bound by the waves of CTAs: 1 .. 6 rows of 16 requests
// in 4 layers of 8 heads of 128, blocks of 64, are 1024 CTAs of 512 threads, 304 of them at a time,
// and each second one returns after it has read a length (7.6 us in a graph).
// APPEND_MANY: the CTAs, 16 rounds of those that an SM holds, from which on LOOP pays; one prompt of
// 2048 tokens in 4 layers of 8 heads of 128 takes 17.8 us with it and 13.1 without.
constexpr int APPEND_MANY = 16 * 4 * 152;
template <int HD, int BLOCK, int U, bool LOOP, typename T>
__global__ void __launch_bounds__(BLOCK* HD / 16, 1024 / (BLOCK * HD / 16))
    append_quant_kernel(CacheArgs c, RowsArgs rows, const int* seq_lens, const int* n_commit,
                        int n_extra, int n_max, int stride) {
  pdl_enter();
  constexpr int THREADS = BLOCK * HD / 16, WARPS = THREADS / 32;
  __shared__ unsigned red[U][WARPS];
  const int h = blockIdx.x % c.heads;
  const int b = blockIdx.y, l = blockIdx.z;
  const int at = seq_lens[b];
  const int64_t n = (int64_t)(n_commit ? n_commit[b] : 0) + n_extra;
  if (!rows_fit(at, n, n_max, c.capacity, c.errors,
                blockIdx.x == 0 && l == 0 && threadIdx.x == 0))
    return;
  if (n == 0) return;
  const int end = at + (int)n, last = (end - 1) / BLOCK;  // the slot behind the rows, their last block

  const int t = threadIdx.x / (HD / 16), d = threadIdx.x % (HD / 16) * 16;
  const int64_t unit = ((int64_t)(c.layer0 + l) * c.batch + b) * c.heads + h;
  const int64_t row0 = l * rows.layer + b * rows.batch + h * rows.head + d;
  for (int first = at / BLOCK + (int)(blockIdx.x / c.heads) * (U / 2); first <= last; first += stride) {
    // what this thread's slot of a unit is: a new row, a committed one, or neither
    auto fresh = [&](int u) {
      const int slot = (first + u / 2) * BLOCK + t;
      return slot >= at && slot < end;
    };
    auto old = [&](int u) { return (first + u / 2) * BLOCK + t < at; };
    auto code = [&](int u) {
      return (u & 1 ? c.v : c.k) + (unit * c.capacity + (first + u / 2) * BLOCK + t) * HD + d;
    };
    auto scale = [&](int u) {
      return (u & 1 ? c.v_scale : c.k_scale) + unit * (c.capacity / BLOCK) + first + u / 2;
    };

    Piece<T> x[U];
    float was[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      was[u] = 0.f;
      if (fresh(u)) {
        const int64_t row = (first + u / 2) * BLOCK + t - at;
        x[u].load(reinterpret_cast<const T*>(u & 1 ? rows.v : rows.k) + row0 + row * rows.token);
      } else if (u < 2 && old(u)) {
        was[u] = *scale(u);
        x[u].u[0] = *reinterpret_cast<const uint4*>(code(u));
      }
    }
    // Magnitudes as bits (their order is the magnitudes' order), the largest over the CTA.
    auto cta_top = [&](int u, unsigned top) {
      top = __reduce_max_sync(0xffffffffu, top);
      if ((threadIdx.x & 31) == 0) red[u][threadIdx.x >> 5] = top;
    };
    auto all_top = [&](int u) {
      unsigned top = red[u][threadIdx.x % WARPS];
#pragma unroll
      for (int o = WARPS / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      return top;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      unsigned top = 0;
      if (fresh(u)) {
        top = x[u].row_top();
      } else if (u < 2 && old(u)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = x[u].code_pair(i, was[u]);
          top = max(top, max(magnitude(f.x), magnitude(f.y)));
        }
      }
      cta_top(u, top);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (first + u / 2 > last) break;
      unsigned top = all_top(u);
      const bool special = top >= 0x7f800000u;
      if (special) {  // (all of the CTA) infinities or NaN: once more without them
        __syncthreads();
        top = 0;
        if (fresh(u) || (u < 2 && old(u))) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = fresh(u) ? x[u].row_pair(i) : x[u].code_pair(i, was[u]);
            top = max(top, max(finite(magnitude(f.x)), finite(magnitude(f.y))));
          }
        }
        cta_top(u, top);
        __syncthreads();
        top = all_top(u);
      }
      // adding 0x1fffff carries into the exponent when the fraction is above 1.75's
      int e = (int)((top + 0x1fffffu) >> 23) - 127 - 8;
      e = top ? min(max(e, -40), 120) : 0;
      const float s = __uint_as_float((unsigned)(127 + e) << 23);
      const float inv = __uint_as_float((unsigned)(127 - e) << 23);
      if (fresh(u) || (u < 2 && old(u) && s != was[u])) {
        uint32_t q[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float2 y[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            y[j] = fresh(u) ? x[u].row_pair(2 * w + j) : x[u].code_pair(2 * w + j, was[u]);
            y[j].x *= inv, y[j].y *= inv;
            if (special) {  // (the conversion saturates: an infinity would become 448)
              if (magnitude(y[j].x) == 0x7f800000u) y[j].x = NAN;
              if (magnitude(y[j].y) == 0x7f800000u) y[j].y = NAN;
            }
          }
          q[w] = (uint32_t)cvt_f32x2_e4m3x2(y[0].x, y[0].y) |
                 (uint32_t)cvt_f32x2_e4m3x2(y[1].x, y[1].y) << 16;
        }
        *reinterpret_cast<uint4*>(code(u)) = make_uint4(q[0], q[1], q[2], q[3]);
      }
      if (threadIdx.x == 0) *scale(u) = s;
    }
    if (!LOOP) break;
    __syncthreads();  // (red is free again)
  }
}

__global__ void __launch_bounds__(256)
    advance_kernel(int batch, int* seq_lens, const int* n_commit, int n_extra, int n_max,
                   int capacity) {
  pdl_enter();
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b >= batch) return;
  const int at = seq_lens[b];
  const int64_t n = (int64_t)(n_commit ? n_commit[b] : 0) + n_extra;
  if (rows_fit(at, n, n_max, capacity, nullptr, false)) seq_lens[b] = at + (int)n;
}

// The committed slots of each request's open block to `saved` or back, with the block's scale: codes
// [k, v][layers][batch slots][heads][block][head_dim], then scales [k, v][layers][batch slots][heads].
// A CTA takes one (layer, request, head)'s keys or values: 16 KB at most, so the call is bound by its
// launch.
template <bool RESTORE>
__global__ void __launch_bounds__(128)
    open_block_kernel(CacheArgs c, int layers, int block, int hd, const int* seq_lens, char* saved) {
  pdl_enter();
  const int h = blockIdx.x % c.heads, b = blockIdx.y, l = c.layer0 + blockIdx.z;
  const bool value = blockIdx.x / c.heads;
  const int at = seq_lens[b];
  if (at < 0 || at > c.capacity) {
    if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0)
      raise_error(c.errors, PEAGLE_DEV_KV_OVERFLOW);
    return;
  }
  const int n = at % block;
  if (n == 0) return;
  const int64_t unit = ((int64_t)l * c.batch + b) * c.heads + h;
  const int64_t units = (int64_t)layers * c.batch * c.heads, kept = (value ? units : 0) + unit;
  uint4* code = reinterpret_cast<uint4*>((value ? c.v : c.k) + (unit * c.capacity + at - n) * hd);
  uint4* code_kept = reinterpret_cast<uint4*>(saved + kept * block * hd);
  float* scale = (value ? c.v_scale : c.k_scale) + unit * (c.capacity / block) + at / block;
  float* scale_kept = reinterpret_cast<float*>(saved + 2 * units * block * hd) + kept;
  for (int i = threadIdx.x; i < n * hd / 16; i += 128)
    if (RESTORE)
      code[i] = code_kept[i];
    else
      code_kept[i] = code[i];
  if (threadIdx.x == 0) {
    if (RESTORE)
      *scale = *scale_kept;
    else
      *scale_kept = *scale;
  }
}

// 16 bytes of row elements from 16 / sizeof(T) codes (packed, low byte first).
__device__ __forceinline__ uint4 decode(const uint2 c, float s, const bf16*) {
  uint32_t r[4];
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = cvt_e4m3x2_f32x2((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
    const __nv_bfloat162 p = __floats2bfloat162_rn(f.x * s, f.y * s);
    r[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ uint4 decode(const uint32_t c, float s, const float*) {
  const float2 a = cvt_e4m3x2_f32x2((uint16_t)c), b = cvt_e4m3x2_f32x2((uint16_t)(c >> 16));
  return make_uint4(__float_as_uint(a.x * s), __float_as_uint(a.y * s), __float_as_uint(b.x * s),
                    __float_as_uint(b.y * s));
}

template <typename T>
struct Codes;
template <>
struct Codes<bf16> {
  typedef uint2 type;
};
template <>
struct Codes<float> {
  typedef uint32_t type;
};

constexpr int READ_THREADS = 256, READ_UNROLL = 4;
// CTAs (8 an SM are in flight) from which on LOOP pays: there are a quarter as many then, and fewer
// find their request shorter than the longest.  16 requests of 1024 .. 8192 slots in 4 layers of 8
// heads of 128 take 264 us with it and 269 without, to fp32 446 and 474; one of 4096 in 4 layers of 8
// heads of 64 10.5 and 9.7.
constexpr int READ_MANY = 16 * 8 * 152;

// A CTA reads READ_THREADS x READ_UNROLL pieces of one (layer, request, kv head), keys or values, and
// with LOOP those `stride` rows further on too: a piece is 16 bytes of row elements, so every store is
// a full one and consecutive threads' loads and stores are consecutive.  Bound by memory: 16 requests
// of 1024 .. 8192 slots in 4 layers of 8 heads of 128 to bf16 take 264 us, 6.86 TB/s (101 % of the
// measured copy rate), to fp32 446 us (100 %); 4096 slots of one in 4 layers of 8 heads of 64 9.7 us
// (76 %) and 15.1 (82 %) in a graph.
template <int HD, bool LOOP, typename T>
__global__ void __launch_bounds__(READ_THREADS)
    read_quant_kernel(CacheArgs c, RowsArgs rows, int block_shift, const int* starts,
                      const int* counts, int n_max, int stride) {
  pdl_enter();
  typedef typename Codes<T>::type Code;
  constexpr int E = 16 / sizeof(T), PER_ROW = HD / E;
  const int h = blockIdx.x % c.heads, rest = blockIdx.x / c.heads;
  const bool value = rest & 1;
  const int b = blockIdx.y, l = blockIdx.z;
  const int at = starts ? starts[b] : 0, n = counts[b];
  if (!rows_fit(at, n, n_max, c.capacity, c.errors,
                blockIdx.x == 0 && l == 0 && threadIdx.x == 0))
    return;
  const int64_t unit = ((int64_t)(c.layer0 + l) * c.batch + b) * c.heads + h;
  const uint8_t* code = (value ? c.v : c.k) + (unit * c.capacity + at) * HD;
  const float* scale = (value ? c.v_scale : c.k_scale) + unit * (c.capacity >> block_shift);
  T* out = reinterpret_cast<T*>(value ? rows.v : rows.k) + l * rows.layer + b * rows.batch +
           h * rows.head;
  // (a thread's pieces are ROWS rows apart, in the same column)
  constexpr int ROWS = READ_THREADS / PER_ROW;
  const int col = threadIdx.x % PER_ROW;
  for (int64_t base = (rest >> 1) * (ROWS * READ_UNROLL); base < n; base += stride) {
    const int row = (int)base + (int)threadIdx.x / PER_ROW;
    const Code* from = reinterpret_cast<const Code*>(code) + (int64_t)row * PER_ROW + col;
    Code got[READ_UNROLL];
    float s[READ_UNROLL];
#pragma unroll
    for (int i = 0; i < READ_UNROLL; ++i) {
      if (row + i * ROWS < n) {
        got[i] = from[i * READ_THREADS];
        s[i] = scale[(at + row + i * ROWS) >> block_shift];
      }
    }
    T* to = out + row * rows.token + col * E;
#pragma unroll
    for (int i = 0; i < READ_UNROLL; ++i, to += ROWS * rows.token)
      if (row + i * ROWS < n) *reinterpret_cast<uint4*>(to) = decode(got[i], s[i], (const T*)nullptr);
    if (!LOOP) break;
  }
}

static int check_rows(const peagle_kv_rows* r) {
  if (!r || !r->k || !r->v) return PEAGLE_ERR_INVALID;
  if (r->dtype != PEAGLE_F32 && r->dtype != PEAGLE_BF16) return PEAGLE_ERR_UNSUPPORTED;
  const int64_t e = r->dtype == PEAGLE_F32 ? 4 : 8;
  if (!aligned(r->k, 16) || !aligned(r->v, 16) || r->layer_stride % e || r->batch_stride % e ||
      r->token_stride % e || r->head_stride % e)
    return PEAGLE_ERR_INVALID;
  return PEAGLE_OK;
}

static CacheArgs cache_args(const peagle_kv_quant* kv, int layer) {
  CacheArgs c;
  c.k = (uint8_t*)kv->k, c.v = (uint8_t*)kv->v;
  c.k_scale = kv->k_scale, c.v_scale = kv->v_scale, c.errors = kv->errors;
  c.batch = kv->batch, c.heads = kv->n_kv_heads, c.capacity = kv->capacity;
  c.layer0 = layer < 0 ? 0 : layer;
  return c;
}

static RowsArgs rows_args(const peagle_kv_rows* r) {
  return RowsArgs{(char*)r->k, (char*)r->v, r->layer_stride, r->batch_stride, r->token_stride,
                  r->head_stride};
}

template <int HD, int BLOCK>
static cudaError_t launch_append(int dtype, int units, bool loop, dim3 grid, cudaStream_t s,
                                 const CacheArgs& c, const RowsArgs& r, const int* seq_lens,
                                 const int* n_commit, int n_extra, int n_max, int stride) {
  auto go = [&](void (*kernel)(CacheArgs, RowsArgs, const int*, const int*, int, int, int)) {
    return launch_pdl(kernel, grid, dim3(BLOCK * HD / 16), 0, s, c, r, seq_lens, n_commit, n_extra,
                      n_max, stride);
  };
  if (dtype == PEAGLE_F32)
    return go(loop ? append_quant_kernel<HD, BLOCK, 2, true, float>
                   : append_quant_kernel<HD, BLOCK, 2, false, float>);
  if (units == 2) return go(append_quant_kernel<HD, BLOCK, 2, false, bf16>);
  return go(loop ? append_quant_kernel<HD, BLOCK, 4, true, bf16>
                 : append_quant_kernel<HD, BLOCK, 4, false, bf16>);
}

}  // namespace kvq
}  // namespace peagle

using namespace peagle;
using namespace peagle::kvq;

extern "C" int peagle_append_kv_quant(const peagle_kv_quant* kv, int32_t layer, int32_t batch,
                                      int32_t* seq_lens, const int32_t* n_commit, int32_t n_extra,
                                      const peagle_kv_rows* rows, int32_t n_max, int32_t advance,
                                      void* stream) {
  int rc = check_cache(kv, layer, batch);
  if (rc != PEAGLE_OK) return rc;
  rc = check_rows(rows);
  if (rc != PEAGLE_OK) return rc;
  if (!seq_lens || seq_lens == n_commit || n_max < 1 || n_max > (1 << 30) || n_extra < -n_max ||
      n_extra > n_max || (advance != 0 && advance != 1))
    return PEAGLE_ERR_INVALID;
  cudaStream_t s = (cudaStream_t)stream;
  const int layers = layer < 0 ? kv->n_layers : 1;
  // the blocks that n_max rows can touch, wherever the first of them starts
  const int64_t blocks = ((int64_t)n_max + kv->block - 2) / kv->block + 1;
  // more than a few blocks a request: four units a CTA (fp32 rows have as many bytes in flight with
  // two)
  const int units = blocks <= 4 || rows->dtype == PEAGLE_F32 ? 2 : 4;
  int64_t ctas = (blocks + units / 2 - 1) / (units / 2);
  const bool loop = blocks > 4 && ctas * kv->n_kv_heads * batch * layers > APPEND_MANY;
  if (loop) ctas = (ctas + 3) / 4;
  const int64_t gx = ctas * kv->n_kv_heads;
  const int stride = (int)(ctas * (units / 2));
  if (gx > INT32_MAX) return PEAGLE_ERR_INVALID;
  const dim3 grid((unsigned)gx, (unsigned)batch, (unsigned)layers);
  const CacheArgs c = cache_args(kv, layer);
  const RowsArgs r = rows_args(rows);
  cudaError_t e = cudaErrorInvalidValue;
#define PEAGLE_APPEND(HD, BLOCK)                                                          \
  if (kv->head_dim == HD && kv->block == BLOCK)                                           \
    e = launch_append<HD, BLOCK>(rows->dtype, units, loop, grid, s, c, r, seq_lens, n_commit,  \
                                 n_extra, n_max, stride);
  PEAGLE_APPEND(64, 16)
  PEAGLE_APPEND(64, 32)
  PEAGLE_APPEND(64, 64)
  PEAGLE_APPEND(64, 128)
  PEAGLE_APPEND(128, 16)
  PEAGLE_APPEND(128, 32)
  PEAGLE_APPEND(128, 64)
  PEAGLE_APPEND(128, 128)
#undef PEAGLE_APPEND
  if (e == cudaSuccess && advance)
    e = launch_pdl(advance_kernel, dim3((unsigned)cdiv(batch, 256)), dim3(256), 0, s, batch,
                   seq_lens, n_commit, n_extra, n_max, kv->capacity);
  return e == cudaSuccess ? PEAGLE_OK : PEAGLE_ERR_CUDA;
}

extern "C" int64_t peagle_save_kv_quant_bytes(const peagle_kv_quant* kv) {
  const int rc = check_cache(kv, -1, 1);
  if (rc != PEAGLE_OK) return rc;
  const int64_t units = (int64_t)kv->n_layers * kv->batch * kv->n_kv_heads;
  // (a cache of this many units fits no GPU, and the bytes no 63 bits)
  if (units > (int64_t)1 << 40) return PEAGLE_ERR_UNSUPPORTED;
  return 2 * units * ((int64_t)kv->block * kv->head_dim + (int64_t)sizeof(float));
}

template <bool RESTORE>
static int open_block(const peagle_kv_quant* kv, int32_t layer, int32_t batch,
                      const int32_t* seq_lens, const void* saved, int64_t saved_bytes,
                      void* stream) {
  const int rc = check_cache(kv, layer, batch);
  if (rc != PEAGLE_OK) return rc;
  if (!seq_lens || !saved || !aligned(saved, 16)) return PEAGLE_ERR_INVALID;
  const int64_t need = peagle_save_kv_quant_bytes(kv);
  if (need < 0) return (int)need;
  if (saved_bytes < need) return PEAGLE_ERR_CAPACITY;
  const dim3 grid(2u * kv->n_kv_heads, (unsigned)batch, layer < 0 ? (unsigned)kv->n_layers : 1u);
  const cudaError_t e =
      launch_pdl(open_block_kernel<RESTORE>, grid, dim3(128), 0, (cudaStream_t)stream,
                 cache_args(kv, layer), kv->n_layers, kv->block, kv->head_dim, seq_lens, (char*)saved);
  return e == cudaSuccess ? PEAGLE_OK : PEAGLE_ERR_CUDA;
}

extern "C" int peagle_save_kv_quant(const peagle_kv_quant* kv, int32_t layer, int32_t batch,
                                    const int32_t* seq_lens, void* saved, int64_t saved_bytes,
                                    void* stream) {
  return open_block<false>(kv, layer, batch, seq_lens, saved, saved_bytes, stream);
}

extern "C" int peagle_restore_kv_quant(const peagle_kv_quant* kv, int32_t layer, int32_t batch,
                                       const int32_t* seq_lens, const void* saved,
                                       int64_t saved_bytes, void* stream) {
  return open_block<true>(kv, layer, batch, seq_lens, saved, saved_bytes, stream);
}

extern "C" int peagle_read_kv_quant(const peagle_kv_quant* kv, int32_t layer, int32_t batch,
                                    const int32_t* starts, const int32_t* counts,
                                    const peagle_kv_rows* out, int32_t n_max, void* stream) {
  int rc = check_cache(kv, layer, batch);
  if (rc != PEAGLE_OK) return rc;
  rc = check_rows(out);
  if (rc != PEAGLE_OK) return rc;
  if (!counts || out->k == out->v || n_max < 1 || n_max > (1 << 30)) return PEAGLE_ERR_INVALID;
  const bool f32 = out->dtype == PEAGLE_F32;
  // n_max rows' pieces; counts are on the device
  const int64_t pieces = (int64_t)n_max * kv->head_dim / (f32 ? 4 : 8);
  const int64_t per = READ_THREADS * READ_UNROLL;
  const int layers = layer < 0 ? kv->n_layers : 1;
  int64_t ctas = (pieces + per - 1) / per;
  const bool loop = ctas * 2 * kv->n_kv_heads * batch * layers > READ_MANY;
  if (loop) ctas = (ctas + 3) / 4;
  const int64_t gx = ctas * 2 * kv->n_kv_heads;
  if (gx > INT32_MAX) return PEAGLE_ERR_INVALID;
  const dim3 grid((unsigned)gx, (unsigned)batch, (unsigned)layers);
  const CacheArgs c = cache_args(kv, layer);
  const RowsArgs r = rows_args(out);
  const int shift = kv->block == 16 ? 4 : kv->block == 32 ? 5 : kv->block == 64 ? 6 : 7;
  const int stride = (int)(ctas * (per * (f32 ? 4 : 8) / kv->head_dim));  // rows, about n_max
  auto launch = [&](void (*kernel)(CacheArgs, RowsArgs, int, const int*, const int*, int, int)) {
    return launch_pdl(kernel, grid, dim3(READ_THREADS), 0, (cudaStream_t)stream, c, r, shift,
                      starts, counts, n_max, stride);
  };
  cudaError_t e = cudaErrorInvalidValue;
#define PEAGLE_READ(HD, LOOP, F32, T) \
  if (kv->head_dim == HD && loop == LOOP && f32 == F32) e = launch(read_quant_kernel<HD, LOOP, T>);
  PEAGLE_READ(64, false, false, bf16)
  PEAGLE_READ(64, true, false, bf16)
  PEAGLE_READ(64, false, true, float)
  PEAGLE_READ(64, true, true, float)
  PEAGLE_READ(128, false, false, bf16)
  PEAGLE_READ(128, true, false, bf16)
  PEAGLE_READ(128, false, true, float)
  PEAGLE_READ(128, true, true, float)
#undef PEAGLE_READ
  return e == cudaSuccess ? PEAGLE_OK : PEAGLE_ERR_CUDA;
}
