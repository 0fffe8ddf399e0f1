// Decode attention over the 8-bit KV cache on the 5th-generation tensor cores, for calls with many
// query rows a kv head (the mathematics, the shares and the second step: kv_quant_attn.cu).
//
// A CTA (one an SM) walks its share in tiles of 128 slots.  Per tile
//   S^T = K Q^T   tcgen05.mma M = 128 slots, N = query rows, K = head_dim, into one of two tensor
//                 memory buffers, so that the next tile's scores are computed during this softmax
//   weights       a thread has one slot: its block's scales are two numbers of the thread, the rows'
//                 references come from shared memory; w = 2^(s + log2 c - m) in f16
//   O += P V      tcgen05.mma M = 128 (query rows, 64 of them used), N = head_dim, K = 128 slots;
//                 both operands lie slot by slot in shared memory (MN-major), as the weights are
//                 made and the values stored; O stays in tensor memory for the whole head
// Slots are the rows of S because decode has few query rows: every thread of the softmax has work
// whatever their number, and the scales need no shuffles.  Codes are converted to f16 (exact) on
// the way from the copied tile to the operands' 128-byte swizzled layout: the 8-bit form of the
// product would need the weights in 8 bits, as two parts of 4 bits for bf16's accuracy.
//
// Warps: 8 softmax (two groups, a half of the query rows each, x four lane quarters of tensor
// memory), 4 converters, one that issues bulk copies of the codes into a ring, one that issues the
// products.  All of them walk the same tiles and hand over through mbarriers, with bounded waits;
// after one that ran out all leave, and the call's error word says so.
//
// The references move as in the warps' kernel: when some weight of a tile would pass 2^LIM, all rows
// of the group move up to the tile's maxima (one vote of its 128 threads a tile), and O is scaled in
// tensor memory after the product before: a group's rows are one quarter's lanes.
//
// What bounds it: the softmax warps' chain of a tile, about 2,600 cycles at 64 rows and head_dim 64
// (the tile's bytes would take 700 at the copy rate, the two products 550), spread over loads from
// tensor memory, 130 arithmetic instructions, the vote, exponentials, and stores with their proxy
// fence; the tensor pipe is 12 % busy.  Two requests of 65536 slots at head_dim 128, 64 rows: 93 us,
// 2.9 TB/s (43 % of the measured copy rate); the warps' kernel takes 158.  Tried and slower: groups
// of 128 threads that each convert, multiply and weigh their own tiles (195 us for what takes 146),
// the weights computed while the votes come in (123 for 108: the code leaves the instruction cache).
#include <atomic>

#include "kv_quant_attn.cuh"

namespace peagle {
namespace kvq {

namespace {

constexpr int TT = 128;        // slots a tile
constexpr int TC_ENTRY = 3;    // what a head costs besides its tiles, in tiles
constexpr int NC = 32;         // query rows a softmax thread
constexpr int TMEM_COLS = 256; // O in columns 0 .. 127, the scores' buffers at 128 and 192
constexpr float SHIFT = SHIFT_BF16;
typedef Segment<TT> TSeg;

// A CTA's warps, in this order: softmax, converters, copies, products.  14 of them leave 128 registers
// a thread; with 8 converters, or 16 softmax warps of 16 rows each, the same calls took 8 .. 20 %
// longer.
constexpr int SOFT = 256, CONV = 128, LOAD_WARP = (SOFT + CONV) / 32, MMA_WARP = LOAD_WARP + 1;
constexpr int WARPS = LOAD_WARP + 2;
constexpr int RP = 64;         // query rows of a part, padded: two groups of softmax warps

// Shared memory of a CTA.
template <int HD>
struct Smem {
  static constexpr int NK = HD == 64 ? 2 : 1;   // f16 key tiles, and query tiles
  static constexpr int NR = HD == 64 ? 5 : 2;   // copied tiles
  static constexpr int F16 = TT * HD * 2, PB = TT * 128, QB = RP * HD * 2, RAW = 2 * TT * HD;
  // (the weights' rows 64 .. 127 are whatever lies a tile further on: the keys behind the second)
  static constexpr int P = 0, K = P + 2 * PB, V = K + NK * F16, Q = V + 2 * F16, R = Q + NK * QB;
  static constexpr int BYTES = R + NR * RAW + 1024;  // (aligned to 1024)
};

// What the warps know of a tile: the copying thread walks the share and leaves this in a ring for
// the others (DESCS entries; nobody is more than NR + 4 tiles behind it).
struct TileDesc {
  int slot, len, b, h;
  int flags;       // FIRST of its head here, LAST, the head BEGAN here, is WHOLE here, END of all
  int piece_slot;  // where the head's tiles begin here
  int chain;       // the CTA of the head's last tile
  int head;        // its number here
};
enum { FIRST = 1, LAST = 2, BEGAN = 4, WHOLE = 8, END = 16 };
constexpr int DESCS = 16;

// The waits that peagle_set_wait_limit_quant can make unreachable (the copies' own completion is
// not one of them: what is in flight has to be waited for).
enum Wait { RAW_EMPTY, K_FULL, V_FULL, S_FULL, S_EMPTY, P_FULL, PV_DONE, HEAD_IN, O_FREE, WAITS };
constexpr unsigned long long DEFAULT_WAIT_NS = 2000000000ull;
std::atomic<unsigned long long> wait_limit{DEFAULT_WAIT_NS};
std::atomic<int> unreachable{-1};

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Whether x holds for any of the threads that meet at the barrier.
__device__ __forceinline__ bool any_of(int id, int threads, bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"((uint32_t)x), "r"(id), "r"(threads)
      : "memory");
  return y != 0;
}
__device__ __forceinline__ float warp_max_f32(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Bytes that a phase of `bar` waits for, without arriving.
__device__ __forceinline__ void expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(tc::smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

// The end of a wait that does not succeed at once (out of line: the code of the loops stays small).
__device__ __noinline__ void wait_long(uint64_t* bar, uint32_t parity, volatile int* abort,
                                       int* errors, unsigned long long limit_ns) {
  if (!tc::mbar_wait(bar, parity, abort, limit_ns)) {
    if (!*abort) raise_error(errors, PEAGLE_DEV_TIMEOUT);
    *abort = 1;
  }
}

// Descriptor of a 128-byte-swizzled operand: 8-row groups 1024 B apart, and, for operands that lie
// MN-major, blocks of 64 M (or N) elements `lbo` bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, int lbo) {
  return (tc::smem_desc_sw128(addr) & ~((uint64_t)0x3fff << 16)) | (uint64_t)(lbo >> 4) << 16;
}

// 16 codes as 16 f16 values.
__device__ __forceinline__ void convert16(uint4 c, uint4& lo, uint4& hi) {
  cvt_e4m3x4_f16x2(c.x, lo.x, lo.y);
  cvt_e4m3x4_f16x2(c.y, lo.z, lo.w);
  cvt_e4m3x4_f16x2(c.z, hi.x, hi.y);
  cvt_e4m3x4_f16x2(c.w, hi.z, hi.w);
}
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
  return w & ~((nan_codes(w) >> 7) * 0xffu);
}

// Sums over the warp's lanes of 32 values a lane: lane i gets the sum of v[i].
__device__ __forceinline__ float scatter_sum(float* v, int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return v[0];
}

template <int HD>
__global__ void __launch_bounds__(WARPS * 32, 1) attn_quant_tc_kernel(AttnQuantArgs a) {
  typedef Smem<HD> M;
  constexpr int NK = M::NK, NR = M::NR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t raw_full[NR], raw_empty[NR], k_full[NK], v_full[2], s_full[2], s_empty[2],
      p_full[2], pv_done[2], head_in, o_free, finished;
  __shared__ uint32_t tmem_at;
  __shared__ volatile int s_abort;
  __shared__ __align__(16) TileDesc descs[DESCS];
  __shared__ __align__(16) float neg_ref[RP], factor[RP], moved[RP];
  __shared__ float tops[4][RP], sums[4][RP];
  __shared__ float scales[DESCS][2 * TT / 16];  // of 16 slots each: keys, then values
  __shared__ float q_scale[4];
  __shared__ __align__(4) uint8_t row_j[2 * RP], bad_row[4][RP];
  __shared__ bool has_slot[RP];
  __shared__ int nan_slots[4];
  __shared__ unsigned conv_top[4][CONV / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int parts = a.heads / a.nkv;
  if (tid < parts * RP) {
    const int of = tid / RP * a.part_rows + tid % RP;
    row_j[tid] = (uint8_t)min(of / a.G, a.K - 1);
  }
  pdl_enter();
  TSeg seg;
  int n;
  int lo, share;
  if (!find_share<TT, TC_ENTRY>(a, 2, seg, n, lo, share)) {
    if (tid == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  if (tid == 0) {
    s_abort = 0;
    auto init = [&](uint64_t* bar, int count, Wait w) { tc::mbar_init(bar, count + (a.stall == w)); };
    for (int i = 0; i < NR; ++i) {
      tc::mbar_init(&raw_full[i], 1);
      init(&raw_empty[i], CONV / 32, RAW_EMPTY);
    }
    for (int i = 0; i < NK; ++i) init(&k_full[i], CONV / 32, K_FULL);
    for (int i = 0; i < 2; ++i) {
      init(&v_full[i], CONV / 32, V_FULL);
      init(&s_full[i], 1, S_FULL);
      init(&s_empty[i], SOFT / 32, S_EMPTY);
      init(&p_full[i], SOFT / 32, P_FULL);
      init(&pv_done[i], 1, PV_DONE);
    }
    init(&head_in, SOFT / 32, HEAD_IN);
    init(&o_free, SOFT / 32, O_FREE);
    tc::mbar_init(&finished, 1);
    tc::fence_barrier_init();
  }
  if (warp == MMA_WARP) {
    tc::tmem_alloc(&tmem_at, TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_at;
  auto wait = [&](uint64_t* bar, int phase) {
    if (!tc::mbar_try_wait(bar, (uint32_t)phase & 1u))
      wait_long(bar, (uint32_t)phase & 1u, &s_abort, a.errors, a.wait_ns);
  };

  int copied = 0;  // tiles that the copying warp issued
  if (warp == LOAD_WARP) {
    // ---- the walk over the share, bulk copies of the codes, and the scales
    const uint64_t policy = tc::policy_evict_first();
    int t = 0, head = 0, u = max(seg.at, 0);
    for (bool more = true; more; ++head) {
      const int end = min(seg.at + seg.tiles, n), u0 = u;
      const int64_t unit = (int64_t)seg.b * a.nkv + seg.h / parts;
      TileDesc d;
      d.len = seg.len, d.b = seg.b, d.h = seg.h, d.head = head;
      d.piece_slot = (seg.first_tile + u0 - seg.at) * TT;
      d.chain = (int)((lo + seg.at + seg.tiles - 1) / share);
      const int base = (seg.at >= 0 ? BEGAN : 0) | (seg.at >= 0 && seg.at + seg.tiles <= n ? WHOLE : 0);
      const int any_begin = row_begin(a, seg.len, 0), any_end = row_end(a, seg.len, a.K - 1);
      const float* from = (lane < 8 ? a.k_scale : a.v_scale) + unit * (a.capacity >> a.block_shift);
      TSeg next = seg;
      more = next.next(a, n);
      bool stop = false;
      for (; u < end; ++u, ++t) {
        d.slot = (seg.first_tile + u - seg.at) * TT;
        d.flags = base | (u == u0 ? FIRST : 0) | (u + 1 == end ? LAST : 0) |
                  (u + 1 == end && !more ? END : 0);
        const int r = t % NR;
        if (t >= NR) wait(&raw_empty[r], t / NR - 1);
        stop = __any_sync(0xffffffffu, s_abort);
        if (stop) break;
        if (lane == 0) {
          // (the capacity may end in the tile)
          const uint32_t bytes = (uint32_t)min(TT, a.capacity - d.slot) * HD;
          uint8_t* to = sm + M::R + r * M::RAW;
          const int64_t at = (unit * a.capacity + d.slot) * HD;
          expect_tx(&raw_full[r], 2 * bytes);
          tc::bulk_load(to, a.k + at, bytes, &raw_full[r], policy);
          tc::bulk_load(to + TT * HD, a.v + at, bytes, &raw_full[r], policy);
          descs[t % DESCS] = d;
        }
        if (lane < 2 * TT / 16) {
          // (scales of blocks without a slot to see may be anything)
          const int x = d.slot + lane % (TT / 16) * 16;
          const bool in = x + 16 > any_begin && x < any_end;
          scales[t % DESCS][lane] = in ? from[x >> a.block_shift] : lane < 8 ? 0.f : 1.f;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&raw_full[r]);
      }
      if (stop) break;
      seg = next;
      u = seg.at;
    }
    copied = t;
    __syncwarp();
  } else if (warp == MMA_WARP) {
    // ---- the products
    if (lane == 0) {
      constexpr uint32_t id_s = (1u << 4) | (uint32_t)(RP >> 3) << 17 | (uint32_t)(TT >> 4) << 24;
      // both operands MN-major
      constexpr uint32_t id_o =
          (1u << 4) | 1u << 15 | 1u << 16 | (uint32_t)(HD >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
      const uint32_t base = tc::smem_u32(sm);
      int flags = 0;  // of the last tile whose scores were issued
      auto scores = [&](int t) {
        if (t >= 2) wait(&s_empty[t & 1], (t - 2) >> 1);
        wait(&k_full[t % NK], t / NK);
        if (s_abort) return;
        tc::fence_after_sync();
        flags = descs[t % DESCS].flags;
        const uint64_t dk = operand_desc(base + M::K + t % NK * M::F16, 16);
        const uint64_t dq = operand_desc(base + M::Q + descs[t % DESCS].head % NK * M::QB, 16);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)
          tc::mma_bf16(tmem + 128 + (t & 1) * 64, dk + (k / 4) * (TT * 128 >> 4) + 2 * (k % 4),
                       dq + (k / 4) * (RP * 128 >> 4) + 2 * (k % 4), id_s, k > 0);
        tc::mma_commit(&s_full[t & 1]);
      };
      scores(0);
      for (int t = 0, heads = 0; !s_abort; ++t) {
        const int mine = flags;
        if (!(mine & END)) scores(t + 1);
        wait(&v_full[t & 1], t >> 1);
        wait(&p_full[t & 1], t >> 1);
        if (mine & FIRST) {
          if (heads > 0) wait(&o_free, heads - 1);
          ++heads;
        }
        if (s_abort) break;
        tc::fence_after_sync();
        const uint64_t dp = operand_desc(base + M::P + (t & 1) * M::PB, M::PB);
        const uint64_t dv = operand_desc(base + M::V + (t & 1) * M::F16, TT * 128);
#pragma unroll
        for (int k = 0; k < TT / 16; ++k)
          tc::mma_bf16(tmem, dp + 128 * k, dv + 128 * k, id_o, !(mine & FIRST) || k > 0);
        tc::mma_commit(&pv_done[t & 1]);
        if (mine & END) break;
      }
      // every product issued is done before tensor memory is freed
      volatile int never = 0;
      tc::mma_commit(&finished);
      tc::mbar_wait(&finished, 0, &never);
    }
    __syncwarp();
  } else if (warp >= SOFT / 32) {
    // ---- converters: queries, keys and values as swizzled f16 operands
    const int ct = tid - SOFT;
    constexpr int QP = RP * HD / 8, QN = (QP + CONV - 1) / CONV;  // 16-byte pieces of a head's queries
    // This thread's 16-byte pieces of a tile: rows ROWS apart (a multiple of 8: the swizzle is the
    // same), ITEMS of them.
    constexpr int ROWS = CONV / (HD / 16), ITEMS = TT / ROWS;
    const int row0 = ct / (HD / 16), c0 = ct % (HD / 16);
    const uint32_t src0 = ct * 16;
    const uint32_t dst0 = c0 / 4 * (TT * 128) + row0 * 128 + ((2 * (c0 % 4) ^ (row0 & 7)) << 4);
    auto convert = [&](const uint8_t* src, uint8_t* dst) {
      uint4 x[ITEMS];  // (all loads before the first store: the compiler may not reorder them)
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        x[i] = *reinterpret_cast<const uint4*>(src + src0 + i * CONV * 16);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        uint4 lo16, hi16;
        convert16(x[i], lo16, hi16);
        *reinterpret_cast<uint4*>(dst + dst0 + i * ROWS * 128) = lo16;
        *reinterpret_cast<uint4*>(dst + (dst0 ^ 16) + i * ROWS * 128) = hi16;
      }
    };
    for (int t = 0;; ++t) {
      const int r = t % NR;
      wait(&raw_full[r], t / NR);
      const TileDesc d = descs[t % DESCS];
      if (t >= NK) wait(&s_full[(t - NK) & 1], (t - NK) >> 1);
      if (any_of(2, CONV, s_abort)) break;  // (all converters or none: they meet at a barrier)
      if (d.flags & FIRST) {
        // One power of two for the head's queries: the largest element to 2^14 .. 2^15.  bf16's 8
        // bits fit f16 down to 2^-31 of it.  Rows that are not finite are told apart and cleared.
        const int at = d.head & 3, part = d.h % parts;
        uint4 raw[QN];
#pragma unroll
        for (int i = 0; i < QN; ++i) {
          const int id = ct + i * CONV, row = id / (HD / 8), of = part * a.part_rows + row;
          raw[i] = make_uint4(0, 0, 0, 0);
          if (row < a.part_rows && of < a.K * a.G) {
            const int j = of / a.G;
            raw[i] = *reinterpret_cast<const uint4*>(
                (const bf16*)a.q + ((int64_t)d.b * a.K + j) * a.q_stride +
                (int64_t)(d.h / parts * a.G + of - j * a.G) * HD + id % (HD / 8) * 8);
          }
        }
        for (int i = ct; i < RP; i += CONV) bad_row[at][i] = 0;
        if (ct == 0) nan_slots[at] = 0;
        unsigned top = 0, bad = 0;
#pragma unroll
        for (int i = 0; i < QN; ++i) {
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const unsigned x = w[k] << 16 & 0x7fffffffu, y = w[k] & 0x7fff0000u;
            if (max(x, y) >= 0x7f800000u) bad |= 1u << i;
            top = max(top, x >= 0x7f800000u ? 0u : x);
            top = max(top, y >= 0x7f800000u ? 0u : y);
          }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) conv_top[at][ct >> 5] = top;
        asm volatile("bar.sync 2, %0;" ::"n"(CONV) : "memory");
#pragma unroll
        for (int i = 0; i < CONV / 32; ++i) top = max(top, conv_top[at][i]);
        const int e = min(max((int)(top >> 23) - 127 - 14, -100), 120);
        const float inv = __uint_as_float((unsigned)(127 - e) << 23);
        if (ct == 0) q_scale[at] = __uint_as_float((unsigned)(127 + e) << 23) * a.scale;
#pragma unroll
        for (int i = 0; i < QN; ++i) {
          const int id = ct + i * CONV, row = id / (HD / 8), c = id % (HD / 8);
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            h[k] = bad >> i & 1 ? 0u
                                : pack_f16(__uint_as_float(w[k] << 16) * inv,
                                           __uint_as_float(w[k] & 0xffff0000u) * inv);
          if (id >= QP) break;
          if (bad >> i & 1) bad_row[at][row] = 1;
          *reinterpret_cast<uint4*>(sm + M::Q + d.head % NK * M::QB + c / 8 * (RP * 128) + row * 128 +
                                    ((c % 8 ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      const uint8_t* from = sm + M::R + r * M::RAW;
      uint8_t* to = sm + M::K + t % NK * M::F16;
      convert(from, to);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&k_full[t % NK]);
      if (t >= 2) wait(&pv_done[t & 1], (t - 2) >> 1);
      to = sm + M::V + (t & 1) * M::F16;
      from += TT * HD;
      const int all_begin = row_begin(a, d.len, a.K - 1), all_end = row_end(a, d.len, 0);
      if (d.slot < all_begin || d.slot + TT > all_end) {
        // Some row does not see some of the tile, and a zero weight does not keep a NaN value out:
        // slots that not all rows see are cleared of NaN, which the rows that see them get back
        // when they are written out.
        bool nan = false;
#pragma unroll 1
        for (int i = 0; i < ITEMS; ++i) {
          const int x = d.slot + row0 + i * ROWS;
          if (x >= all_begin && x < all_end) continue;
          uint4* p = reinterpret_cast<uint4*>(const_cast<uint8_t*>(from) + src0 + i * CONV * 16);
          const uint4 w = *p;
          if (nan_codes(w.x) | nan_codes(w.y) | nan_codes(w.z) | nan_codes(w.w)) {
            *p = make_uint4(without_nan(w.x), without_nan(w.y), without_nan(w.z), without_nan(w.w));
            nan = true;
          }
        }
        if (nan) nan_slots[d.head & 3] = 1;
      }
      convert(from, to);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&v_full[t & 1]);
        tc::mbar_arrive(&raw_empty[r]);
      }
      if (d.flags & END) break;
    }
  } else {
    // ---- softmax: this thread's slot of every tile, NC query rows from column col0 on
    const int quarter = warp & 3, part32 = warp >> 2, col0 = part32 * NC;
    const int key = quarter * 32 + lane;  // (of this group's 128 threads too)
    const int bar = 3 + part32;
    auto group_any = [&](bool x) { return any_of(bar, 128, x); };
    auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory"); };
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    float l[NC];
    bool pending, chained = false, stop = false;
    auto new_head = [&]() {
      if (key < NC) neg_ref[col0 + key] = 0.f, has_slot[col0 + key] = false;
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = 0.f;
      pending = true;
      group_sync();
    };
    new_head();
    for (int t = 0; !stop; ++t) {
      const int b = t & 1;
      wait(&s_full[b], t >> 1);
      // (of no meaning after an abort: nothing up to the vote that ends the loop then may make some of
      // the group's threads meet at a barrier and not others)
      const TileDesc d = descs[t % DESCS];
      tc::fence_after_sync();
      float x[NC];
      tc::tmem_ld32(tmem + lanes + 128 + b * 64 + col0, x);
      tc::tmem_ld_wait();
      const float vs = scales[t % DESCS][TT / 16 + key / 16];
      const float g = scales[t % DESCS][key / 16] * q_scale[d.head & 3], lv = lg2(vs);
      const float rv = inverse_scale(vs);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s_empty[b]);
#pragma unroll
      for (int c = 0; c < NC; c += 4) {
        const float4 m = *reinterpret_cast<const float4*>(&neg_ref[col0 + c]);
        x[c] = fmaf(x[c], g, lv + m.x), x[c + 1] = fmaf(x[c + 1], g, lv + m.y);
        x[c + 2] = fmaf(x[c + 2], g, lv + m.z), x[c + 3] = fmaf(x[c + 3], g, lv + m.w);
      }
      if (d.slot < row_begin(a, d.len, a.K - 1) || d.slot + TT > row_end(a, d.len, 0)) {
        // the draft rows that see this thread's slot
        const int over = d.slot + key - d.len;
        const int j0 = a.causal ? over : over < 0 ? 0 : a.K, j1 = a.window > 0 ? over + a.window - 1 : a.K;
        // (unsigned: in row_j whatever a descriptor that a wait ran out on holds)
        const unsigned part = (unsigned)d.h % (unsigned)parts;
        const uint32_t* rows = reinterpret_cast<const uint32_t*>(row_j + part * RP + col0);
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const uint32_t w = rows[c / 4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = w >> (8 * k) & 0xff;
            if (j < j0 || j > j1) x[c + k] = -INFINITY;
          }
        }
      }
      float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < NC; c += 2) top4[c / 2 % 4] = max3(top4[c / 2 % 4], x[c], x[c + 1]);
      const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
      // (NaN passes no comparison: it reaches the weights as it is)
      if (group_any(top > LIM || pending || s_abort)) {
        stop = group_any(s_abort);
        if (stop) break;
        float mine = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float y = warp_max_f32(x[c]);
          if (lane == c) mine = y;
        }
        tops[quarter][col0 + lane] = mine;
        group_sync();
        bool missing = false;
        if (key < NC) {
          const int c = col0 + key;
          const float y = fmaxf(fmaxf(tops[0][c], tops[1][c]), fmaxf(tops[2][c], tops[3][c]));
          const bool any = !(y == -INFINITY), had = has_slot[c];
          const float by = !any ? 0.f : had ? fmaxf(y - SHIFT, 0.f) : y - SHIFT;
          factor[c] = had ? ex2(-by) : 1.f;
          moved[c] = -by;
          neg_ref[c] -= by;
          has_slot[c] = had || any;
          missing = !(had || any);
        }
        pending = group_any(missing);
        if (!(d.flags & FIRST) && quarter == part32) {
          // the group's rows are the lanes of this quarter of tensor memory
          wait(&pv_done[b ^ 1], (t - 1) >> 1);
          tc::fence_after_sync();
          const float f = factor[col0 + lane];
#pragma unroll 1
          for (int i = 0; i < HD; i += 16) {
            const uint32_t to = tmem + lanes + i;
            float o[16];
            tc::tmem_ld16(to, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] *= f;
            asm volatile(
                "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(to),
                "f"(o[0]), "f"(o[1]), "f"(o[2]), "f"(o[3]), "f"(o[4]), "f"(o[5]), "f"(o[6]),
                "f"(o[7]), "f"(o[8]), "f"(o[9]), "f"(o[10]), "f"(o[11]), "f"(o[12]), "f"(o[13]),
                "f"(o[14]), "f"(o[15])
                : "memory");
          }
          tc::tmem_st_wait();
        }
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&factor[col0 + c]);
          const float4 y = *reinterpret_cast<const float4*>(&moved[col0 + c]);
          l[c] *= f.x, l[c + 1] *= f.y, l[c + 2] *= f.z, l[c + 3] *= f.w;
          x[c] += y.x, x[c + 1] += y.y, x[c + 2] += y.z, x[c + 3] += y.w;
        }
      }
      uint32_t p[NC / 2];
#pragma unroll
      for (int c = 0; c < NC; c += 2) {
        const float w0 = ex2(x[c]), w1 = ex2(x[c + 1]);
        l[c] = fmaf(w0, rv, l[c]), l[c + 1] = fmaf(w1, rv, l[c + 1]);
        p[c / 2] = pack_f16(w0, w1);
      }
      if (t >= 2) wait(&pv_done[b], (t - 2) >> 1);
      uint8_t* to = sm + M::P + b * M::PB + key * 128;
#pragma unroll
      for (int i = 0; i < NC / 8; ++i)
        *reinterpret_cast<uint4*>(to + ((part32 * (NC / 8) + i ^ (key & 7)) << 4)) =
            make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
      fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&p_full[b]);

      if (d.flags & LAST) {
        // ---- the head's result, or this CTA's piece of it
        const float sum = scatter_sum(l, lane);
        sums[quarter][col0 + lane] = sum;
        wait(&pv_done[b], t >> 1);
        // (waits and not barriers between the groups: after an abort one may not come)
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&head_in);
        wait(&head_in, d.head);
        tc::fence_after_sync();
        const int row = quarter * 32 + lane;
        const bool began = d.flags & BEGAN, whole = d.flags & WHOLE;
        if (quarter * 32 < RP) {
          const int part = d.h % parts, kvh = d.h / parts, of = part * a.part_rows + row;
          const bool exists = row < a.part_rows && of < a.K * a.G;
          const int j = of / a.G;
          float sum_l = 1.f, m = NO_REF, inv = 0.f;
          bf16* out = nullptr;
          float* work = a.work + ((size_t)blockIdx.x * 2 + (began ? 1 : 0)) * (RP * (HD + 2));
          if (row < RP) {
            m = has_slot[row] ? -neg_ref[row] : NO_REF;
            sum_l = sums[0][row] + sums[1][row] + sums[2][row] + sums[3][row];
            if (bad_row[d.head & 3][row] && has_slot[row]) sum_l = NAN;
            if (!whole && part32 == 0) *reinterpret_cast<float2*>(work + 2 * row) = make_float2(m, sum_l);
          }
          if (whole && exists)
            out = finish_row<bf16>(a, HD, d.b, j * (a.nkv * a.G) + kvh * a.G + of - j * a.G, m, sum_l,
                                   part32 == 0, inv);
          const bool patch = nan_slots[d.head & 3] && exists;
#pragma unroll 1
          for (int i0 = part32 * 16; i0 < HD; i0 += 32) {
            float o[16];
            tc::tmem_ld16(tmem + lanes + i0, o);
            tc::tmem_ld_wait();
            if (patch) {
              // NaN values of slots that only some rows see, among this piece's tiles
              const int begin = max(row_begin(a, d.len, j), d.piece_slot);
              const int end = min(row_end(a, d.len, j), d.slot + TT);
              const int all_begin = row_begin(a, d.len, a.K - 1), all_end = row_end(a, d.len, 0);
              for (int y = begin; y < end; ++y) {
                if (y >= all_begin && y < all_end) {
                  y = all_end - 1;
                  continue;
                }
                const uint4 v = *reinterpret_cast<const uint4*>(
                    a.v + (((int64_t)d.b * a.nkv + kvh) * a.capacity + y) * HD + i0);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (nan_codes(w[i / 4]) >> (8 * (i % 4)) & 0x80) o[i] = NAN;
              }
            }
            if (out) {
              uint32_t h[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const __nv_bfloat162 z = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
                h[k] = *reinterpret_cast<const uint32_t*>(&z);
              }
              reinterpret_cast<uint4*>(out + i0)[0] = make_uint4(h[0], h[1], h[2], h[3]);
              reinterpret_cast<uint4*>(out + i0)[1] = make_uint4(h[4], h[5], h[6], h[7]);
            } else if (!whole && row < RP) {
              float4* to_o = reinterpret_cast<float4*>(work + 2 * RP + row * HD + i0);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                to_o[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
          }
        }
        if (began && !whole) {
          chained = true;
          if (tid == 0) a.desc[blockIdx.x] = make_int4(d.b, d.h, d.chain, 0);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&o_free);
        wait(&o_free, d.head);  // (the references and sums are free again)
        new_head();
      }
      if (d.flags & END) break;
    }
    if (tid == 0 && !chained) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, TMEM_COLS);
  }
  if (warp == LOAD_WARP && lane == 0 && s_abort) {
    // The copies in flight, whoever gave up and however long after the last of them was issued.
    volatile int never = 0;
    for (int x = max(0, copied - NR); x < copied; ++x)
      tc::mbar_wait(&raw_full[x % NR], (uint32_t)(x / NR) & 1u, &never);
  }
}

template <int HD>
cudaError_t launch(const AttnQuantArgs& a, cudaStream_t s) {
  const size_t smem = Smem<HD>::BYTES;
  auto kernel = attn_quant_tc_kernel<HD>;
  cudaError_t e = smem_optin((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(CTAS), dim3(WARPS * 32), smem, s, a);
  if (e != cudaSuccess) return e;
  return launch_join(HD, false, true, a, RP / 8, s);
}

}  // namespace

// Where this kernel takes less time than the warps' one (us, this one against that one; slots = the
// slots of all requests and kv heads):
//   head_dim 128, 64 rows:  1048576 slots 93 / 158, 262144 37 / 53, 131072 27 / 33, 65536 21.5 / 23.6
//   head_dim 128, 40 rows:  1048576 slots 92 / 141, 262144 36 / 48, 131072 26 / 29, 65536 20.6 / 21.6
//   head_dim 64, 64 rows:   1048576 slots 76 / 83, 524288 45 / 48, 262144 29.4 / 29.7, 131072 22 / 21
//   head_dim 64, 40 rows:   1048576 slots 76 / 72
//   head_dim 64, 64 rows, 64 requests of 300 .. 4100 slots: 93 / 108
// Its chain of a tile is longer (conversion, product, softmax, product), so it wants several tiles a
// CTA; and below 33 rows half of its softmax threads would have none.
bool attn_quant_tc_takes(int hd, bool f32, int rows, int64_t slots) {
  return !f32 && rows > (hd == 64 ? 48 : 32) &&
         slots * cdiv(rows, RP) >= (hd == 64 ? 3 : 1) << 16;
}

// (more than 32 rows, whatever the slots; parts are equal up to one row)
int attn_quant_tc_rows(int rows) { return rows > 32 ? RP : 0; }

cudaError_t launch_attention_tc(int hd, int rows, AttnQuantArgs a, cudaStream_t s) {
  const int parts = cdiv(rows, RP);
  a.part_rows = cdiv(rows, parts);
  a.heads = a.nkv * parts;
  a.wait_ns = wait_limit.load(), a.stall = unreachable.load();
  return hd == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace kvq
}  // namespace peagle

extern "C" int peagle_set_wait_limit_quant(uint64_t limit_ns, int32_t unreachable_wait) {
  using namespace peagle::kvq;
  if (unreachable_wait < -1 || unreachable_wait >= WAITS) return PEAGLE_ERR_INVALID;
  wait_limit.store(limit_ns ? (unsigned long long)limit_ns : DEFAULT_WAIT_NS);
  unreachable.store(unreachable_wait);
  return PEAGLE_OK;
}
