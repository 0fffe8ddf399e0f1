// Decode attention over the 8-bit KV cache: peagle_decode_attention_quant.
//
// The draft block's attention ("P-EAGLE: A Technical Deep Dive into Parallel Speculative
// Decoding", section "2. The P-EAGLE Parallel Drafter": the K rows of a request attend over
// the cache and the rows before them), reading codes and block scales.
//
// Mathematics.  With codes k, v and scales a, c of a slot's block, and everything in the log2
// domain, s = (q . k) a scale log2(e), and
//     out = sum_t 2^s_t c_t v_t / sum_t 2^s_t.
// The kernel holds, for each row, a reference m and sums the weights w_t = 2^(s_t + log2 c_t - m):
//     O = sum_t w_t v_t (codes, on the tensor cores),   l = sum_t w_t / c_t,   out = O / l,
// so a value's scale rides in the exponential's argument and weights of quiet and loud blocks
// alike lie where the tensor operand's 11 bits are.  m moves only when a weight would pass 2^LIM
// (and O and l are scaled then), which after the first tiles is rare.  Sums and statistics are
// fp32.
//
// Tensor work: m16n8k16 with f16 operands, keys (then head dims) as the 16 rows and the query
// rows as the 8 columns, because a decode batch has few query rows.  Codes become f16 exactly
// (one conversion instruction for two); the e4m3 form of the instruction is no faster here, it
// runs as conversions and f16 products (0.43 an SM and clock measured with changing operands,
// for twice the depth of an f16 one at 0.48).
//   S^T = K Q^T  bf16 queries, each row scaled by a power of two, are exact in f16; fp32 queries
//                come as two f16 parts.
//   O^T = V^T P  a weight keeps 11 bits; for fp32 queries it is two f16 parts.
// The contraction's order over head dims is free, so a lane takes 16 consecutive bytes of a
// key for its K operand; the order of the output's head dims is free, so a lane takes 8 or 16
// consecutive bytes of 4 keys for V^T and pairs them with byte permutes: no transposes in shared
// memory.
//
// Work split.  A unit is a tile of 32 slots of one (request, kv head).  All units of the call,
// in order, are cut into equal consecutive shares, one for each of CTAS CTAs (one an SM), so
// ragged batches and single long requests fill the GPU alike.  Inside a CTA W / groups streams
// of warps take the tiles of a (request, kv head) in turn (groups of warps share a stream's
// tiles when there are more query rows than one warp's registers hold), each with its own
// cp.async ring in shared memory that runs on across (request, kv head) boundaries.  At the end
// of one its streams are joined in shared memory; one that lies whole in a CTA is written out,
// pieces of one go to the workspace and the second kernel joins them.
// Calls with short heads take one step instead: every (request, kv head) belongs to a cluster of
// 1 .. 8 CTAs, which cut its tiles among them and join their results through one another's shared
// memory (split_of).
#include "kv_quant_attn.cuh"

namespace peagle {
namespace kvq {

constexpr int TILE = 32;       // slots a unit
constexpr int ENTRY = 28;      // see find_share; 24 and 32 measured within 2 %, 8 up to 20 % slower
constexpr int MAX_SPLIT = 8;   // CTAs of a cluster that share a head
typedef Segment<TILE> Seg;

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum: zeros as C, which take no registers.
__device__ __forceinline__ void mma_f16_first(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// (the remaining 4 - bytes are zeros)
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Wait until at most `pending` of the newest groups are in flight.
__device__ __forceinline__ void cp_async_wait(int pending) {
  switch (pending) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
  }
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(p));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
  return v;
}

// (an address that mapa_shared gave)
__device__ __forceinline__ float4 ld_cluster(uint32_t p) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(p)
               : "memory");
  return v;
}

// Byte offset of 16-byte chunk `chunk` of row `row` in a tile of rows of HD bytes.  The chunks
// of a 128-byte line are permuted by bits of the row so that both readers are free of bank
// conflicts: a phase of the K operand's loads takes 4 chunks of rows 2i and 2i + 1, one of the
// V operand's the same 2 chunks of rows 0, 2, 4, 6 (or 1, 3, 5, 7).
template <int HD>
__device__ __forceinline__ uint32_t tile_offset(int row, int chunk) {
  if (HD == 128) {
    const int f = ((row ^ (row >> 2)) & 1) << 2 | (row & 2);
    return (uint32_t)(row * 128 + ((chunk ^ f) << 4));
  }
  const int line = row >> 1;
  return (uint32_t)(line * 128 + ((((row & 1) << 2 | chunk) ^ ((line & 3) << 1)) << 4));
}

__device__ __forceinline__ float power2(int e) {
  return __uint_as_float((unsigned)(127 + e) << 23);
}

// A lane's query elements: 16 consecutive ones of row 8 tile + r at head dims 16c and, for
// head_dim 128, 64 + 16c, as they are stored (zeros past the last row).
template <int HD, bool F32>
struct RawQuery {
  static constexpr int E = F32 ? 4 : 8, N = HD / 4 / E;
  uint4 u[N];

  __device__ __forceinline__ void fetch(const AttnQuantArgs& a, int req, int h, int tile,
                                        int lane) {
    const int row = tile * 8 + (lane >> 2), c = lane & 3;
    if (row < a.K * a.G) {
      const int j = row / a.G;
      const char* q = (const char*)a.q +
                      (((int64_t)req * a.K + j) * a.q_stride +
                       (int64_t)(h * a.G + row - j * a.G) * HD + 16 * c) * (F32 ? 4 : 2);
#pragma unroll
      for (int i = 0; i < N; ++i)
        u[i] = *reinterpret_cast<const uint4*>(
            q + ((i * E / 16) * 64 + i * E % 16) * (F32 ? 4 : 2));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] = make_uint4(0, 0, 0, 0);
    }
  }
  // The elements, and the largest magnitude of the row as bits.
  __device__ __forceinline__ unsigned elements(float* x) const {
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (F32) {
          x[E * i + k] = __uint_as_float(w[k]);
        } else {
          x[E * i + 2 * k] = __uint_as_float(w[k] << 16);
          x[E * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < HD / 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    return max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  }
};

template <int HD, int NT, bool F32>
struct Queries {
  static constexpr int STEPS = HD / 16, PARTS = F32 ? 2 : 1;
  static constexpr int TILE_BYTES = PARTS * STEPS * 32 * 8;
  uint32_t b[PARTS][STEPS][NT][2];  // [part][k step][rows][register]
  float scale[NT][2];               // of rows 2c and 2c + 1, with the scores' scale

  __device__ __forceinline__ static void prepare(const RawQuery<HD, F32>& raw, float scale,
                                                 int lane, uint2* to, float* scales) {
    float x[HD / 4];
    const unsigned top = raw.elements(x);
    const bool fine = top < 0x7f800000u;
    // the largest element to 2^14 .. 2^15: f16's last bit is then 2^-38 of it
    const int e = fine ? min(max((int)(top >> 23) - 127 - 14, -100), 120) : 0;
    const float inv = power2(-e);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      uint32_t part[PARTS][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float y0 = x[4 * s + 2 * i] * inv, y1 = x[4 * s + 2 * i + 1] * inv;
        part[0][i] = pack_f16(y0, y1);
        const float2 f = unpack_f16(part[0][i]);
        if (F32) part[PARTS - 1][i] = pack_f16(y0 - f.x, y1 - f.y);
      }
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        to[(p * STEPS + s) * 32 + lane] = make_uint2(part[p][0], part[p][1]);
    }
    // a row that is not finite gives NaN
    if ((lane & 3) == 0) scales[lane >> 2] = fine ? power2(e) * scale : NAN;
  }

  __device__ __forceinline__ void load(const uint2* from, const float* scales, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const uint2 u = from[nt * (TILE_BYTES / 8) + (p * STEPS + s) * 32 + lane];
          b[p][s][nt][0] = u.x, b[p][s][nt][1] = u.y;
        }
      const float2 f = reinterpret_cast<const float2*>(scales)[nt * 4 + (lane & 3)];
      scale[nt][0] = f.x, scale[nt][1] = f.y;
    }
  }

  // acc[nt] = the scores of 16 keys (rows 0 .. 15 from shared address k).  `off`: the lane's
  // first chunk.
  __device__ __forceinline__ void scores(float (*acc)[4], uint32_t k, uint32_t off) const {
#pragma unroll
    for (int half = 0; half < HD / 64; ++half) {
      // (chunk c + 4 of a 128-byte row is chunk c with its bit 2 flipped)
      const uint4 u4 = lds128(k + (off ^ (half * 64)));
      const uint4 w4 = lds128(k + (off ^ (half * 64)) + 8 * HD);
      const uint32_t u[4] = {u4.x, u4.y, u4.z, u4.w}, w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t a0, a1, a2, a3;
        cvt_e4m3x4_f16x2(u[s], a0, a2);
        cvt_e4m3x4_f16x2(w[s], a1, a3);
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (half == 0 && s == 0 && p == 0)
              mma_f16_first(acc[nt], a0, a1, a2, a3, b[0][0][nt][0], b[0][0][nt][1]);
            else
              mma_f16(acc[nt], a0, a1, a2, a3, b[p][4 * half + s][nt][0],
                      b[p][4 * half + s][nt][1]);
          }
      }
    }
  }
};

// One warp's running result over a (request, kv head): NT x 8 query rows.  O^T's fragment: head
// dim r HD / 8 + 2 i (elements 0, 1) and the next one (2, 3), rows 2c (0, 2) and 2c + 1 (1, 3).
template <int HD, int NT, bool F32>
struct Running {
  static constexpr float SHIFT = F32 ? SHIFT_F32 : SHIFT_BF16;
  float o[HD / 16][NT][4];
  float m[NT][2], l[NT][2];
  unsigned started;  // bit 2 nt + e: the row has seen a slot (its m counts)

  __device__ __forceinline__ void clear() {
    started = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = 0.f;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.f;
    }
  }

  // A tile of 32 slots from `slot` on.  edge: some row does not see some of it.  rows: each query
  // row's draft row.
  __device__ __forceinline__ void tile(const AttnQuantArgs& a, const Queries<HD, NT, F32>& q,
                                       uint32_t k, uint32_t v, uint32_t scales, int slot,
                                       bool edge, int len, const uint8_t* rows, int lane) {
    const int r = lane >> 2, c = lane & 3;
    const uint32_t k_off = tile_offset<HD>(r, c);
    const uint4 sc = lds128(scales);
    float x[2][NT][4];  // the scores, then the weights' exponents
    q.scores(x[0], k, k_off);
    q.scores(x[1], k + 16 * HD, k_off);
    const float ks[2] = {__uint_as_float(sc.x), __uint_as_float(sc.y)};
    // (16 slots without any to see come without scales)
    const float vs[2] = {sc.z ? __uint_as_float(sc.z) : 1.f, sc.w ? __uint_as_float(sc.w) : 1.f};
    const float lv[2] = {lg2(vs[0]), lg2(vs[1])};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const float f0 = q.scale[nt][0] * ks[sub], f1 = q.scale[nt][1] * ks[sub];
        const float g0 = lv[sub] - m[nt][0], g1 = lv[sub] - m[nt][1];
        float* w = x[sub][nt];
        w[0] = fmaf(w[0], f0, g0), w[1] = fmaf(w[1], f1, g1);
        w[2] = fmaf(w[2], f0, g0), w[3] = fmaf(w[3], f1, g1);
      }
    }
    unsigned seen = ~0u;  // bit (sub * NT + nt) * 4 + j: element j's slot is seen by its row
    static_assert(2 * NT * 4 <= 32, "one bit an element");
    if (edge) {
      seen = 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = rows[nt * 8 + 2 * c + e];
          const int lo = row_begin(a, len, j) - slot - r, hi = row_end(a, len, j) - slot - r;
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              if (sub * 16 + y * 8 >= lo && sub * 16 + y * 8 < hi)
                seen |= 1u << ((sub * NT + nt) * 4 + 2 * y + e);
              else
                x[sub][nt][2 * y + e] = -INFINITY;
            }
        }
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        top = max3(top, x[sub][nt][0], x[sub][nt][1]);
        top = max3(top, x[sub][nt][2], x[sub][nt][3]);
      }
    // (NaN passes no comparison: it reaches the weights as it is)
    constexpr unsigned ALL = (1u << (2 * NT)) - 1;
    if (__any_sync(0xffffffffu, top > LIM || started != ALL)) raise(x);
    const float rv[2] = {inverse_scale(vs[0]), inverse_scale(vs[1])};
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      uint32_t p[F32 ? 2 : 1][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* w = x[sub][nt];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = ex2(w[j]);
        l[nt][0] = fmaf(w[0] + w[2], rv[sub], l[nt][0]);
        l[nt][1] = fmaf(w[1] + w[3], rv[sub], l[nt][1]);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t hi = pack_f16(w[2 * y], w[2 * y + 1]);
          p[0][nt][y] = transpose8(hi);
          if (F32) {
            const float2 f = unpack_f16(hi);
            p[F32 ? 1 : 0][nt][y] = transpose8(pack_f16(w[2 * y] - f.x, w[2 * y + 1] - f.y));
          }
        }
      }
      values(p, v + sub * 16 * HD, edge, seen >> (sub * NT * 4), lane);
    }
  }

  // Moves the references of the rows that a tile passes or starts, and scales what was summed.
  __device__ __forceinline__ void raise(float (*x)[NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = fmaxf(max3(x[0][nt][e], x[0][nt][2 + e], x[1][nt][e]), x[1][nt][2 + e]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const bool any = !(top == -INFINITY), had = started >> (2 * nt + e) & 1;
        // (rows below their limit move up too: that is room for later tiles)
        const float by = !any ? 0.f : had ? fmaxf(top - SHIFT, 0.f) : top - SHIFT;
        const float f = had ? ex2(-by) : 1.f;  // (nothing was summed before the first slot)
        if (any) started |= 1u << (2 * nt + e);
        m[nt][e] += by;
        l[nt][e] *= f;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) x[sub][nt][e] -= by, x[sub][nt][2 + e] -= by;
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) o[i][nt][e] *= f, o[i][nt][2 + e] *= f;
      }
    }
  }

  // O^T += V^T P over 16 slots (rows 0 .. 15 from shared address v).
  __device__ __forceinline__ void values(const uint32_t (*p)[NT][2], uint32_t v, bool edge,
                                         unsigned seen, int lane) {
    constexpr int WORDS = HD / 32;  // of a lane's bytes of one slot
    const int r = lane >> 2, c = lane & 3;
    uint32_t w[4][WORDS];  // slots 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int row = 2 * c + (s & 1);  // (8 rows further on the chunks are permuted alike)
      if (HD == 128) {
        const uint4 u = lds128(v + tile_offset<HD>(row, r) + (s >> 1) * 8 * HD);
        w[s][0] = u.x, w[s][1] = u.y, w[s][WORDS - 2] = u.z, w[s][WORDS - 1] = u.w;
      } else {
        const uint2 u = lds64(v + tile_offset<HD>(row, r >> 1) + (r & 1) * 8 + (s >> 1) * 8 * HD);
        w[s][0] = u.x, w[s][1] = u.y;
      }
    }
    if (edge) {
      // A slot that some row does not see may hold NaN, and a zero weight does not keep it out.
      // Its codes are cleared, and the rows that see it are made NaN by a product of the two
      // 0 / 1 matrices "is NaN" and "is seen".
      uint32_t bad = 0;
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < WORDS; ++j) bad |= nan_codes(w[s][j]);
      if (__any_sync(0xffffffffu, bad)) {
        uint32_t one[4][WORDS];  // e4m3 1.0 where a code is NaN
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int j = 0; j < WORDS; ++j) {
            const uint32_t n = nan_codes(w[s][j]) >> 7;
            one[s][j] = n * 0x38u;
            w[s][j] &= ~(n * 0xffu);
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const unsigned bits = seen >> (nt * 4);
          const uint32_t b0 = transpose8((bits & 1 ? 0x3c00u : 0u) | (bits & 2 ? 0x3c000000u : 0u));
          const uint32_t b1 = transpose8((bits & 4 ? 0x3c00u : 0u) | (bits & 8 ? 0x3c000000u : 0u));
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) {
            float n[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t x[4];
            operand(one, i, x);
            mma_f16(n, x[0], x[1], x[2], x[3], b0, b1);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (n[j] > 0.f) o[i][nt][j] = NAN;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < HD / 16; ++i) {
      uint32_t x[4];
      operand(w, i, x);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_f16(o[i][nt], x[0], x[1], x[2], x[3], p[0][nt][0], p[0][nt][1]);
        if (F32)
          mma_f16(o[i][nt], x[0], x[1], x[2], x[3], p[F32 ? 1 : 0][nt][0], p[F32 ? 1 : 0][nt][1]);
      }
    }
  }

  // The V^T operand of head dims r HD / 8 + 2 i, + 1 from a lane's bytes of its four slots.
  __device__ __forceinline__ static void operand(const uint32_t (*w)[HD / 32], int i,
                                                 uint32_t* x) {
    const unsigned sel = i & 1 ? 0x7362u : 0x5140u;  // bytes of two slots, side by side
    const uint32_t a = __byte_perm(w[0][i >> 1], w[1][i >> 1], sel);
    const uint32_t b = __byte_perm(w[2][i >> 1], w[3][i >> 1], sel);
    cvt_e4m3x4_f16x2(a, x[0], x[1]);
    cvt_e4m3x4_f16x2(b, x[2], x[3]);
  }
};

// Warps a CTA: as many as their registers allow, 8 with up to 255 or 12 with 168.  12 read 65536
// slots at head_dim 64 in 93 us for 8 query rows (8 warps 99, 16 warps 89) and 99 for 16 (115, 149);
// 24 rows no longer fit (199 for 134), nor does head_dim 128 gain (8 rows 93 for 94).
constexpr int warps_of(int hd, int nt, bool f32) { return hd == 64 && nt <= 2 && !f32 ? 12 : 8; }

// Parts in which the warps' O^T go through the joining buffer.  At head_dim 128 parts leave room
// for a third stage of the rings (NT 1 and 2; NT 3 has two either way).
constexpr int join_passes(int hd, int nt) { return hd == 64 ? 1 : nt == 2 ? 4 : 2; }

template <int HD, int NT, bool F32, int W>
__global__ void __launch_bounds__(W * 32, 1) attn_quant_kernel(AttnQuantArgs a) {
  typedef typename std::conditional<F32, float, bf16>::type T;
  typedef Queries<HD, NT, F32> Q;
  constexpr int STAGE = 2 * TILE * HD + 16;  // K, V, four scales
  constexpr int FRAG = HD / 16 * NT * 32;    // float4s of a warp's O^T
  constexpr int PASSES = join_passes(HD, NT), PASS = FRAG / PASSES;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(8) float row_m[W][NT * 8], row_l[W][NT * 8];
  __shared__ __align__(8) float row_scale[MAX_ROWS + 8];
  __shared__ float sum_m[MAX_ROWS + 8], sum_l[MAX_ROWS + 8];
  __shared__ uint8_t row_j[MAX_ROWS + 8];  // each query row's draft row
  __shared__ int row_at[MAX_ROWS + 8];     // and place among its request's rows and heads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = a.groups, streams = W / groups;
  const int stream = warp / groups, group = warp % groups;
  const int row0 = group * NT * 8;
  if (threadIdx.x < groups * NT * 8) {
    const int j = min((int)threadIdx.x / a.G, a.K - 1);  // (past the last row: the last draft row)
    row_j[threadIdx.x] = (uint8_t)j;
    row_at[threadIdx.x] = j * (a.nkv * a.G) + (int)threadIdx.x - j * a.G;
  }
  pdl_enter();

  // a share below 4 tiles would leave warps idle and make pieces to join
  Seg seg;
  int n, lo, share;
  if (a.split) {
    lo = share = 0;
    if (!find_heads<HD, T>(a, seg, n)) return;
  } else if (!find_share<TILE, ENTRY>(a, 4, seg, n, lo, share)) {
    if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }

  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) +
                        (uint32_t)(stream * a.stages) * STAGE;
  uint2* prepared = reinterpret_cast<uint2*>(smem + (size_t)streams * a.stages * STAGE);
  float4* joined = reinterpret_cast<float4*>(prepared + groups * NT * (Q::TILE_BYTES / 8));
  float* piece = reinterpret_cast<float*>(joined + W * PASS);  // what the cluster's CTAs join

  // The stream's loads run ahead of its products, over (request, kv head) boundaries.  A lane
  // copies the same chunks of every tile: rows WARP_ROWS groups apart, whose places in a stage
  // follow from two offsets (rows 4 apart are permuted differently, rows 8 apart alike).
  constexpr int ROW_CHUNKS = HD / 16, WARP_ROWS = 32 / ROW_CHUNKS;
  Seg next = seg;
  int next_u = 0, next_end = 0, slot_in = 0;
  const uint8_t *next_k = nullptr, *next_v = nullptr;
  const float* next_scale = nullptr;
  const int my_row = group * WARP_ROWS + lane / ROW_CHUNKS;
  const uint32_t off_even = tile_offset<HD>(my_row, lane % ROW_CHUNKS);
  const uint32_t off_odd = tile_offset<HD>(my_row + WARP_ROWS * groups, lane % ROW_CHUNKS) -
                           WARP_ROWS * groups * HD;
  bool more = true;
  auto enter = [&]() {  // the stream's first tile of segment `next`
    next_u = max(next.at, 0) + stream;
    next_end = min(next.at + next.tiles, n);
    const int64_t unit = (int64_t)next.b * a.nkv + next.h;
    const int64_t slot = (int64_t)(next.first_tile + next_u - next.at) * TILE;
    const int64_t at = (unit * a.capacity + slot + my_row) * HD + lane % ROW_CHUNKS * 16;
    next_k = a.k + at;
    next_v = a.v + at;
    next_scale = (lane < 2 ? a.k_scale : a.v_scale) + unit * (a.capacity >> a.block_shift);
  };
  auto issue = [&]() {
    while (more && next_u >= next_end) {
      more = next.next(a, n);
      if (more) enter();
    }
    if (more) {
      const int slot = (next.first_tile + next_u - next.at) * TILE;
      const uint32_t to = ring + slot_in * STAGE;
      if (my_row >= TILE) {  // (more groups than the tile has rows for)
      } else if (slot + TILE <= a.capacity) {
        for (int i = 0; i < TILE; i += 2 * WARP_ROWS * groups) {
          const int by = WARP_ROWS * groups;
          cp_async16(to + off_even + i * HD, next_k + i * HD);
          cp_async16(to + TILE * HD + off_even + i * HD, next_v + i * HD);
          if (i + by < TILE) {
            cp_async16(to + off_odd + (i + by) * HD, next_k + (i + by) * HD);
            cp_async16(to + TILE * HD + off_odd + (i + by) * HD, next_v + (i + by) * HD);
          }
        }
      } else {  // a tile that the capacity ends in
        for (int i = 0; i < TILE; i += WARP_ROWS * groups) {
          const uint32_t off = tile_offset<HD>(my_row + i, lane % ROW_CHUNKS);
          if (my_row + i < TILE && slot + my_row + i < a.capacity) {
            cp_async16(to + off, next_k + i * HD);
            cp_async16(to + TILE * HD + off, next_v + i * HD);
          }
        }
      }
      if (group == 0 && lane < 4) {
        // (scales of blocks without a slot to see may be anything: zeros instead)
        const int t = slot + (lane & 1) * 16;
        const bool in = t + 16 > row_begin(a, next.len, 0) && t < row_end(a, next.len, a.K - 1);
        cp_async4(to + 2 * TILE * HD + lane * 4, in ? next_scale + (t >> a.block_shift) : a.k_scale,
                  in ? 4 : 0);
      }
      next_u += streams;
      next_k += (int64_t)streams * TILE * HD;
      next_v += (int64_t)streams * TILE * HD;
    }
    cp_async_commit();
    if (++slot_in == a.stages) slot_in = 0;
  };
  enter();
  for (int i = 0; i < a.stages - 1; ++i) issue();

  RawQuery<HD, F32> raw;
  if (warp < groups * NT) raw.fetch(a, seg.b, seg.h, warp, lane);
  Q q;
  Running<HD, NT, F32> run;
  const int r = lane >> 2, c = lane & 3;
  int slot_out = 0;
  bool chained = false;
  while (true) {
    const int begin = max(seg.at, 0), end = min(seg.at + seg.tiles, n);
    const int all_begin = row_begin(a, seg.len, a.K - 1), all_end = row_end(a, seg.len, 0);
    for (int t = warp; t < groups * NT; t += W) {
      if (t >= W) raw.fetch(a, seg.b, seg.h, t, lane);
      Q::prepare(raw, a.scale, lane, prepared + t * (Q::TILE_BYTES / 8), row_scale + t * 8);
    }
    run.clear();
    __syncthreads();
    q.load(prepared + group * NT * (Q::TILE_BYTES / 8), row_scale + row0, lane);
    for (int u = begin + stream; u < end; u += streams) {
      cp_async_wait(a.stages - 2);
      if (groups > 1)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + stream), "r"(32 * groups) : "memory");
      else
        __syncwarp();
      issue();
      const uint32_t at = ring + slot_out * STAGE;
      const int slot = (seg.first_tile + u - seg.at) * TILE;
      const bool edge = slot < all_begin || slot + TILE > all_end;
      run.tile(a, q, at, at + TILE * HD, at + 2 * TILE * HD, slot, edge, seg.len, row_j + row0,
               lane);
      if (++slot_out == a.stages) slot_out = 0;
    }

    // the next (request, kv head)'s queries arrive while this one's streams are joined
    const Seg done = seg;
    const bool last = !seg.next(a, n);
    if (!last && warp < groups * NT) raw.fetch(a, seg.b, seg.h, warp, lane);

    // join the streams: their references, sums and outputs by way of shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1)
          run.l[nt][e] += __shfl_xor_sync(0xffffffffu, run.l[nt][e], d);
        if (r == 0) {
          row_m[warp][nt * 8 + 2 * c + e] = run.started >> (2 * nt + e) & 1 ? run.m[nt][e] : NO_REF;
          row_l[warp][nt * 8 + 2 * c + e] = run.l[nt][e];
        }
      }
    const bool began = done.at >= 0, whole = began && done.at + done.tiles <= n;
    float* slot = a.split > 1 ? piece
                              : a.work + ((size_t)blockIdx.x * 2 + (began ? 1 : 0)) *
                                             ((size_t)groups * NT * 8 * (HD + 2));
    // column i of the fragments of rows row and row + 1
    auto write = [&](int row, int i, float m0, float l0, float m1, float l1, const float4& o) {
      const int d = r * (HD / 8) + 2 * i;
      float inv;
      if (row < a.K * a.G) {
        T* out = finish_row<T>(a, HD, done.b, done.h * a.G + row_at[row], m0, l0,
                               i == 0 && r == 0, inv);
        store2(out + d, o.x * inv, o.z * inv);
      }
      if (row + 1 < a.K * a.G) {
        T* out = finish_row<T>(a, HD, done.b, done.h * a.G + row_at[row + 1], m1, l1,
                               i == 0 && r == 0, inv);
        store2(out + d, o.y * inv, o.w * inv);
      }
    };
#pragma unroll 1
    for (int pass = 0; pass < PASSES; ++pass) {
      if (pass) __syncthreads();
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
        if (i / (HD / 16 / PASSES) == pass)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float* o = run.o[i][nt];
            joined[warp * PASS + (nt * (HD / 16 / PASSES) + i % (HD / 16 / PASSES)) * 32 + lane] =
                make_float4(o[0], o[1], o[2], o[3]);
          }
      __syncthreads();
      if (pass == 0) {
        // each row's common reference and sum, and what each stream's output counts there
        if (threadIdx.x < groups * NT * 8) {
          const int g = threadIdx.x / (NT * 8), row = threadIdx.x % (NT * 8);
          float m = NO_REF, l = 0.f;
          for (int w = g; w < W; w += groups) m = fmaxf(m, row_m[w][row]);
          for (int w = g; w < W; w += groups) {
            const float f = ex2(row_m[w][row] - m);
            l = fmaf(row_l[w][row], f, l);
            row_m[w][row] = f;
          }
          sum_m[threadIdx.x] = m, sum_l[threadIdx.x] = l;
        }
        __syncthreads();
      }
      // each warp sums some of the fragments over the streams
#pragma unroll 1
      for (int at = warp; at < groups * (PASS / 32); at += W) {
        const int g = at / (PASS / 32), in = at % (PASS / 32);
        const int nt = in / (HD / 16 / PASSES), i = pass * (HD / 16 / PASSES) + in % (HD / 16 / PASSES);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = g; w < W; w += groups) {
          const float4 x = joined[w * PASS + in * 32 + lane];
          const float2 f = *reinterpret_cast<const float2*>(&row_m[w][nt * 8 + 2 * c]);
          o.x = fmaf(x.x, f.x, o.x), o.y = fmaf(x.y, f.y, o.y);
          o.z = fmaf(x.z, f.x, o.z), o.w = fmaf(x.w, f.y, o.w);
        }
        const int row = (g * NT + nt) * 8 + 2 * c;
        const float m0 = sum_m[row], m1 = sum_m[row + 1], l0 = sum_l[row], l1 = sum_l[row + 1];
        if (whole && a.split < 2) {
          write(row, i, m0, l0, m1, l1, o);
        } else {
          if (i == 0 && r == 0)
            *reinterpret_cast<float4*>(slot + 2 * row) = make_float4(m0, l0, m1, l1);
          reinterpret_cast<float4*>(
              slot + (size_t)groups * NT * 16)[((g * NT + nt) * (HD / 16) + i) * 32 + lane] = o;
        }
      }
    }
    if (a.split > 1) {
      // the cluster's warps share the columns of the pieces, which they read in one another's memory
      __syncwarp();
      tc::cluster_sync();
      const int cols = groups * NT * (HD / 16);
      for (int col = (int)tc::cluster_ctarank() * W + warp; col < cols; col += a.split * W) {
        const int i = col % (HD / 16), row = col / (HD / 16) * 8 + 2 * c;
        float4 f[MAX_SPLIT], g[MAX_SPLIT];
        float m0 = NO_REF, m1 = NO_REF, l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int p = 0; p < MAX_SPLIT; ++p) {
          f[p] = make_float4(NO_REF, 0.f, NO_REF, 0.f);
          g[p] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (p < a.split) {
            const uint32_t from = tc::mapa_shared(piece, p);
            f[p] = ld_cluster(from + 8 * row);
            g[p] = ld_cluster(from + 64 * groups * NT + 16 * (col * 32 + lane));
          }
        }
#pragma unroll
        for (int p = 0; p < MAX_SPLIT; ++p) m0 = fmaxf(m0, f[p].x), m1 = fmaxf(m1, f[p].z);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p = 0; p < MAX_SPLIT; ++p) {
          const float x0 = ex2(f[p].x - m0), x1 = ex2(f[p].z - m1);
          l0 = fmaf(f[p].y, x0, l0), l1 = fmaf(f[p].w, x1, l1);
          o.x = fmaf(g[p].x, x0, o.x), o.y = fmaf(g[p].y, x1, o.y);
          o.z = fmaf(g[p].z, x0, o.z), o.w = fmaf(g[p].w, x1, o.w);
        }
        write(row, i, m0, l0, m1, l1, o);
      }
      __syncwarp();
      tc::cluster_sync();  // (a CTA's memory is its own again, or may end)
    } else if (began && !whole) {
      chained = true;
      if (threadIdx.x == 0)
        a.desc[blockIdx.x] =
            make_int4(done.b, done.h, (int)((lo + done.at + done.tiles - 1) / share), 0);
    }
    if (last) break;
  }
  if (threadIdx.x == 0 && !chained && !a.split) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
  cp_async_wait(0);
}

// Joins the pieces of the (request, kv head)s that several CTAs worked on: block (c, z) takes the
// one whose first piece CTA c holds, and of its ntiles x HD / 16 columns of 32 fragments the z-th
// 4 / JOIN_WARPS; JOIN_WARPS warps split a column's pieces.  Bound by the latency of the pieces' loads
// (they are in L2), so a warp has up to 8 of them in flight and goes over them once, and by the start
// of the blocks that find nothing to join: four warps a block, whatever the split.  With 8 heads and
// more (about 19 pieces a head at most) one warp a column takes less time, 20 query rows of 16 requests
// 53.1 us with the first kernel for 57.0; one head of 16416 slots 10.4 with four for 16.1.  Also
// writes the rows of requests no row of which sees a slot.  ROWS: outputs lie row by row, a lane's
// float4 is four head dims of one row; else as fragments (struct Running).
template <int HD, typename T, bool ROWS, int JOIN_WARPS>
__global__ void __launch_bounds__(128) attn_quant_join_kernel(AttnQuantArgs a, int ntiles) {
  pdl_enter();
  constexpr int JOIN_COLS = 4 / JOIN_WARPS;
  __shared__ float4 red_o[JOIN_COLS][JOIN_WARPS][32];
  __shared__ float4 red_ml[JOIN_COLS][JOIN_WARPS][32];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % JOIN_WARPS;
  const int sub = threadIdx.x / (32 * JOIN_WARPS);
  const int4 d = a.desc[blockIdx.x];
  if (blockIdx.y == 0) {
    for (int b = blockIdx.x; b < a.batch; b += CTAS) {
      const int len = a.seq_lens[b];
      int first;
      if (!request_fits(a, len) || request_tiles<TILE>(a, len, first)) continue;
      write_empty<HD, T>(a, b, 0, a.nkv);
    }
  }
  if (d.x < 0) return;
  const int col = blockIdx.y * JOIN_COLS + sub;  // (HD / 16 is a multiple of 4)
  const int pieces = d.z - (int)blockIdx.x + 1;
  const size_t slot = (size_t)ntiles * 8 * (HD + 2);
  // (piece p > 0 is the head of CTA c + p's share: slot 0; the first is the tail of c's: slot 1)
  const float* base = a.work + (size_t)blockIdx.x * 2 * slot;
  const int r = lane >> 2, c = lane & 3;
  const int nt = col / (HD / 16), i = col % (HD / 16);
  const int row = ROWS ? (col * 32 + lane) / (HD / 4) : nt * 8 + 2 * c;
  float m0 = NO_REF, m1 = NO_REF, l0 = 0.f, l1 = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int BATCH = 8;
  for (int p0 = warp; p0 < pieces; p0 += BATCH * JOIN_WARPS) {
    float4 f[BATCH], g[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int p = p0 + k * JOIN_WARPS;
      const float* s = base + ((size_t)2 * p + (p == 0 ? 1 : 0)) * slot;
      f[k] = make_float4(NO_REF, 0.f, NO_REF, 0.f);
      g[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p < pieces) {
        if (ROWS) {
          const float2 x = *reinterpret_cast<const float2*>(s + 2 * row);
          f[k] = make_float4(x.x, x.y, x.x, x.y);
        } else {
          f[k] = *reinterpret_cast<const float4*>(s + 2 * row);
        }
        g[k] = reinterpret_cast<const float4*>(s + (size_t)ntiles * 16)[col * 32 + lane];
      }
    }
    float n0 = m0, n1 = m1;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) n0 = fmaxf(n0, f[k].x), n1 = fmaxf(n1, f[k].z);
    float x0 = ex2(m0 - n0), x1 = ex2(m1 - n1);
    l0 *= x0, l1 *= x1;
    o = make_float4(o.x * x0, o.y * x1, o.z * x0, o.w * x1);
    m0 = n0, m1 = n1;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      x0 = ex2(f[k].x - m0), x1 = ex2(f[k].z - m1);
      l0 = fmaf(f[k].y, x0, l0), l1 = fmaf(f[k].w, x1, l1);
      o.x = fmaf(g[k].x, x0, o.x), o.y = fmaf(g[k].y, x1, o.y);
      o.z = fmaf(g[k].z, x0, o.z), o.w = fmaf(g[k].w, x1, o.w);
    }
  }
  if (JOIN_WARPS > 1) {
    red_o[sub][warp][lane] = o;
    red_ml[sub][warp][lane] = make_float4(m0, l0, m1, l1);
    __syncthreads();
    if (warp) return;
    l0 = l1 = 0.f;
    m0 = m1 = NO_REF;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < JOIN_WARPS; ++w)
      m0 = fmaxf(m0, red_ml[sub][w][lane].x), m1 = fmaxf(m1, red_ml[sub][w][lane].z);
#pragma unroll
    for (int w = 0; w < JOIN_WARPS; ++w) {
      const float4 f = red_ml[sub][w][lane], g = red_o[sub][w][lane];
      const float x0 = ex2(f.x - m0), x1 = ex2(f.z - m1);
      l0 = fmaf(f.y, x0, l0), l1 = fmaf(f.w, x1, l1);
      o.x = fmaf(g.x, x0, o.x), o.y = fmaf(g.y, x1, o.y);
      o.z = fmaf(g.z, x0, o.z), o.w = fmaf(g.w, x1, o.w);
    }
  }
  float inv;
  const int nq = a.nkv * a.G;
  if (ROWS) {
    const int parts = a.heads / a.nkv, part = d.y % parts, of = part * a.part_rows + row;
    if (row < a.part_rows && of < a.K * a.G) {
      const int at = (col * 32 + lane) % (HD / 4) * 4, j = of / a.G;
      T* out = finish_row<T>(a, HD, d.x, j * nq + d.y / parts * a.G + of - j * a.G, m0, l0,
                             at == 0, inv);
      store2(out + at, o.x * inv, o.y * inv);
      store2(out + at + 2, o.z * inv, o.w * inv);
    }
  }
  const int j0 = row / a.G, j1 = (row + 1) / a.G;
  if (!ROWS && row < a.K * a.G) {
    T* out = finish_row<T>(a, HD, d.x, j0 * nq + d.y * a.G + row - j0 * a.G, m0, l0,
                           i == 0 && r == 0, inv);
    store2(out + r * (HD / 8) + 2 * i, o.x * inv, o.z * inv);
  }
  if (!ROWS && row + 1 < a.K * a.G) {
    T* out = finish_row<T>(a, HD, d.x, j1 * nq + d.y * a.G + row + 1 - j1 * a.G, m1, l1,
                           i == 0 && r == 0, inv);
    store2(out + r * (HD / 8) + 2 * i, o.y * inv, o.w * inv);
  }
}

// How the query rows of a kv head are laid over warps: groups of warps x NT tiles of 8 rows.
// A warp's registers hold the queries and the outputs of NT tiles: 24 NT registers for
// head_dim 64 (32 NT with fp32 queries), 48 NT (64 NT) for 128.  As many rows a warp as they hold:
// each warp of a group converts the codes for itself.  24 rows over 65536 slots at head_dim 64 take
// 134 us as one group of three tiles and 210 as two groups; 16 warps with half the registers and
// two tiles each took 161 us where 8 with four took 124 (64 rows, a batch of 64).
struct Plan {
  int nt, groups;
  int ntiles() const { return nt * groups; }
};
static Plan plan_of(int hd, bool f32, int rows) {
  const int tiles = cdiv(rows, 8), most = hd == 64 ? 4 : f32 ? 2 : 3;
  Plan p;
  for (p.groups = 1; cdiv(tiles, p.groups) > most; p.groups *= 2) {
  }
  p.nt = cdiv(tiles, p.groups);
  return p;
}

static size_t slot_bytes(int hd, int ntiles) { return (size_t)ntiles * 8 * (hd + 2) * sizeof(float); }
static int64_t work_bytes(int hd, int ntiles) {
  return 4096 + (int64_t)CTAS * 2 * (int64_t)slot_bytes(hd, ntiles);
}

// Clusters of CTAs as large as these that the GPU's GPCs hold at a time.
static int clusters_of(int split) { return split == 1 ? CTAS : split == 2 ? 76 : split == 4 ? 36 : 15; }

// The CTAs that share a head when the call is done in one step, or 0 when two steps take less time
// (equal shares of the call's tiles, and the kernel that joins their pieces).  As many CTAs as find
// room, unless one does the head in a round of its warps.  Two steps spread long and ragged heads
// better, one saves a launch, the way through the workspace and shares that lie over two heads; a
// round's cost follows from its products.  us in one step / in two, requests at full capacity and, in
// brackets, spread from none of it to all:
//   slots a head:           544                       1056                      2080
//   4 rows of 128, 8 heads  7.2 / 11.0                7.6 / 11.6                8.6 / 9.4
//   20 rows of 128, 16      11.5 / 17.1 (10.7 / 17.1) 13.7 / 12.2 (11.6 / 17.0) 15.8 / 13.3 (13.4 / 12.2)
//   20 fp32 rows of 128, 32 13.0 / 13.7 (11.3 / 17.4) 15.1 / 17.5 (13.3 / 13.7) 19.9 / 21.3 (17.1 / 15.8)
//   8 rows of 64, 32        6.6 / 8.2 (6.5 / 10.3)    7.1 / 10.6 (6.9 / 8.2)    8.1 / 10.6 (7.9 / 10.6)
//   64 rows of 64, 8        9.3 / 13.7                10.6 / 14.4               11.8 / 11.6
//   64 rows of 64, 72       12.0 / 14.2 (11.0 / 14.4) 14.4 / 17.1 (13.3 / 14.8) 20.6 / 25.3 (18.1 / 17.1)
//   (4128 slots: 9.9 / 10.3 for the first, 14.4 / 12.9 for 64 rows of 64, 8 heads)
static int split_of(int hd, bool f32, const Plan& p, int warps, int64_t heads, int64_t slots) {
  const int64_t tiles = (slots / TILE + 2) * p.groups;
  int split = tiles <= warps ? 1 : MAX_SPLIT;
  while (heads > clusters_of(split) && split > 1) split /= 2;
  const int64_t per = (heads + clusters_of(split) - 1) / clusters_of(split);  // heads a cluster
  const double round = hd / 64 * (p.nt * (f32 ? 2 : 1) + 2) / 5.;             // us, about
  const double one = (double)tiles / (warps * split);                         // rounds a head
  const double rounds = (double)per * (one + 2) - 2;
  const double shares = (double)heads * (double)tiles / (CTAS * warps);
  const double saved = .3 * p.ntiles() > 1.8 ? .3 * p.ntiles() : 1.8;
  return (rounds - shares) * round <= saved ? split : 0;
}

template <int HD, int NT, bool F32, int W>
static cudaError_t launch_attention(AttnQuantArgs a, const Plan& p, cudaStream_t s) {
  constexpr size_t STAGE = 2 * TILE * HD + 16;
  constexpr size_t JOIN = (size_t)W * HD * NT * 32 / join_passes(HD, NT);
  const int streams = W / p.groups;
  const size_t fixed = JOIN + (size_t)p.ntiles() * Queries<HD, NT, F32>::TILE_BYTES +
                       (a.split > 1 ? slot_bytes(HD, p.ntiles()) : 0);
  // up to 8 stages a stream, within the 227 KB of a CTA less its static arrays
  const size_t room = 221 * 1024 - fixed;
  a.groups = p.groups;
  a.stages = (int)(room / (streams * STAGE));
  a.stages = a.stages > 8 ? 8 : a.stages;
  const size_t smem = streams * a.stages * STAGE + fixed;
  auto kernel = attn_quant_kernel<HD, NT, F32, W>;
  cudaError_t e = smem_optin((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  if (!a.split) {
    e = launch_pdl(kernel, dim3(CTAS), dim3(W * 32), smem, s, a);
    return e == cudaSuccess ? launch_join(HD, F32, false, a, p.ntiles(), s) : e;
  }
  const int64_t heads = (int64_t)a.batch * a.heads, most = clusters_of(a.split);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((heads < most ? heads : most) * a.split));
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_join(int hd, bool f32, bool rowmajor, const AttnQuantArgs& a, int ntiles,
                        cudaStream_t s) {
  const bool many = (int64_t)a.batch * a.heads >= 8;
  auto go = [&](void (*kernel)(AttnQuantArgs, int)) {
    return launch_pdl(kernel, dim3(CTAS, ntiles * (hd / 16) / (many ? 4 : 1)), dim3(128), 0, s, a,
                      ntiles);
  };
#define PEAGLE_JOIN(HD, T, ROWS) \
  go(many ? attn_quant_join_kernel<HD, T, ROWS, 1> : attn_quant_join_kernel<HD, T, ROWS, 4>)
  if (rowmajor) return hd == 64 ? PEAGLE_JOIN(64, bf16, true) : PEAGLE_JOIN(128, bf16, true);
  if (f32) return hd == 64 ? PEAGLE_JOIN(64, float, false) : PEAGLE_JOIN(128, float, false);
  return hd == 64 ? PEAGLE_JOIN(64, bf16, false) : PEAGLE_JOIN(128, bf16, false);
#undef PEAGLE_JOIN
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
  if (K > MAX_ROWS || K * (int64_t)(n_q_heads / kv->n_kv_heads) > MAX_ROWS)
    return PEAGLE_ERR_UNSUPPORTED;
  return PEAGLE_OK;
}

extern "C" int64_t peagle_decode_attention_quant_workspace(const peagle_kv_quant* kv,
                                                           int32_t batch, int32_t K,
                                                           int32_t n_q_heads) {
  const int rc = check_attention(kv, batch, K, n_q_heads);
  if (rc != PEAGLE_OK) return rc;
  const int rows = K * (n_q_heads / kv->n_kv_heads);
  // (the largest of the query types' plans)
  const int a = plan_of(kv->head_dim, false, rows).ntiles();
  const int b = plan_of(kv->head_dim, true, rows).ntiles(), c = attn_quant_tc_rows(rows) / 8;
  const int most = a > b ? a : b;
  return work_bytes(kv->head_dim, most > c ? most : c);
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
      (causal != 0 && causal != 1) || window < 0 || !isfinite(scale * LOG2E))
    return PEAGLE_ERR_INVALID;
  if (dtype != PEAGLE_F32 && dtype != PEAGLE_BF16) return PEAGLE_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) || !aligned(out_lse, 4) ||
      q_stride % (dtype == PEAGLE_F32 ? 4 : 8))
    return PEAGLE_ERR_INVALID;
  if (workspace_bytes < need) return PEAGLE_ERR_CAPACITY;
  // (the walk over the tiles counts in 31 bits; a cache beyond that does not fit a GPU)
  if ((int64_t)batch * kv->n_kv_heads * 2 * (kv->capacity / TILE + 2 + ENTRY) >= 1 << 30)
    return PEAGLE_ERR_UNSUPPORTED;
  const int hd = kv->head_dim;
  const bool f32 = dtype == PEAGLE_F32;
  // (out is written while other heads' queries are still to be read)
  const int64_t size = f32 ? 4 : 2, row = (int64_t)n_q_heads * hd * size, rows = (int64_t)batch * K;
  const int64_t step = q_stride ? q_stride * size : row, apart = step < 0 ? -step : step;
  const int64_t to = (int64_t)(intptr_t)out;
  const int64_t q0 = (int64_t)(intptr_t)q + (step < 0 ? (rows - 1) * step : 0);
  const int64_t first = to - row < q0 ? 0 : (to - row - q0) / apart + 1;  // row that ends behind `to`
  if (first < rows && q0 + first * apart < to + rows * row) return PEAGLE_ERR_INVALID;
  const int64_t unit = (int64_t)layer * kv->batch * kv->n_kv_heads;
  AttnQuantArgs a;
  a.k = (const uint8_t*)kv->k + unit * kv->capacity * hd;
  a.v = (const uint8_t*)kv->v + unit * kv->capacity * hd;
  a.k_scale = kv->k_scale + unit * (kv->capacity / kv->block);
  a.v_scale = kv->v_scale + unit * (kv->capacity / kv->block);
  a.q = q;
  a.q_stride = q_stride ? q_stride : (int64_t)n_q_heads * hd;
  a.out = out, a.lse = out_lse, a.seq_lens = seq_lens, a.errors = kv->errors;
  a.desc = (int4*)workspace;
  a.work = (float*)((char*)workspace + 4096);
  a.batch = batch, a.K = K, a.G = n_q_heads / kv->n_kv_heads, a.nkv = kv->n_kv_heads;
  a.capacity = kv->capacity;
  a.block_shift = kv->block == 16 ? 4 : kv->block == 32 ? 5 : kv->block == 64 ? 6 : 7;
  // (a window that no row's slots reach the end of is none: the kernels add slots to it in 32 bits)
  if (window > kv->capacity + K) window = 0;
  a.causal = causal, a.window = window, a.scale = scale * LOG2E;
  a.heads = a.nkv, a.part_rows = K * a.G;
  // the slots that a head sees at most
  const int64_t most = window > 0 && window < kv->capacity - K ? window + K : kv->capacity;
  const Plan p = plan_of(hd, f32, K * a.G);
  const int warps = warps_of(hd, p.nt, f32);
  const int64_t heads = (int64_t)batch * a.nkv;
  cudaError_t e = cudaErrorInvalidValue;
  // (the tcgen05 kernel only where heads are more than two rounds of a CTA's warps)
  a.split = 0;
  if ((most / TILE + 2) * p.groups > 2 * warps && attn_quant_tc_takes(hd, f32, K * a.G, heads * most))
    return launch_attention_tc(hd, K * a.G, a, (cudaStream_t)stream) == cudaSuccess ? PEAGLE_OK
                                                                                    : PEAGLE_ERR_CUDA;
  a.split = split_of(hd, f32, p, warps, heads, most);
#define PEAGLE_ATTN(HD, NT, F32)                                                           \
  if (hd == HD && p.nt == NT && f32 == F32)                                                \
    e = launch_attention<HD, NT, F32, warps_of(HD, NT, F32)>(a, p, (cudaStream_t)stream);
  PEAGLE_ATTN(64, 1, false)
  PEAGLE_ATTN(64, 2, false)
  PEAGLE_ATTN(64, 3, false)
  PEAGLE_ATTN(64, 4, false)
  PEAGLE_ATTN(64, 1, true)
  PEAGLE_ATTN(64, 2, true)
  PEAGLE_ATTN(64, 3, true)
  PEAGLE_ATTN(64, 4, true)
  PEAGLE_ATTN(128, 1, false)
  PEAGLE_ATTN(128, 2, false)
  PEAGLE_ATTN(128, 3, false)
  PEAGLE_ATTN(128, 1, true)
  PEAGLE_ATTN(128, 2, true)
#undef PEAGLE_ATTN
  return e == cudaSuccess ? PEAGLE_OK : PEAGLE_ERR_CUDA;
}
