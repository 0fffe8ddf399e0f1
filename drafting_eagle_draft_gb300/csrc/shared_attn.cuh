// Attention of a batch over a prefix that all of its requests share and over their own slots behind
// it: what the kernels have in common (entry point and join: shared_attn.cu).
#pragma once

#include "common.cuh"

namespace peagle {
namespace sha {

constexpr int64_t MAX_ROWS = 1 << 24;   // batch * K * heads
constexpr int MAX_SLOTS = 1 << 24;      // of a prefix, of a request

struct Args {
  const void* q;  // [batch * K][nq][hd], rows q_stride apart
  int64_t q_stride;
  const void* pk;  // [nkv][pcap][hd]
  const void* pv;
  const int* prefix_len;  // [1]
  const void* k;          // [batch][nkv][cap][hd]
  const void* v;
  const int* lens;  // [batch]
  int batch, K, nq, nkv, G, pcap, cap, causal;
  float scale;
  void* out;
  float* lse;
  int* errors;
  float* part;  // workspace
  int entry;    // (bf16) what a unit costs besides its tiles
};

// The bf16 kernels (shared_attn_tc.cu).
int64_t tc_workspace(int64_t batch, int K, int G, int nkv, int hd, int pcap, int cap);
int launch_tc(Args a, int hd, cudaStream_t st);

// Slots of the prefix, or -1 where it does not fit.
__device__ __forceinline__ int prefix_of(const Args& a) {
  const int n = *a.prefix_len;
  return n >= 0 && n <= a.pcap ? n : -1;
}
// Slots of request b that its last row sees, or -1 where they do not fit.
__device__ __forceinline__ int slots_of(const Args& a, int b) {
  const int n = a.lens[b];
  if (n < 0 || n > a.cap - (a.causal ? a.K : 0)) return -1;
  return n + (a.causal ? a.K : 0);
}
// Slots that row j of a request sees, of the `slots` that its last row does.
__device__ __forceinline__ int limit_of(const Args& a, int slots, int j) {
  return a.causal ? slots - (a.K - 1 - j) : slots;
}

// A partial result of a row and head: sum of 2^(s - m) v, and m (log2) and the sum of 2^(s - m).
struct Stat {
  float m, l;
};

}  // namespace sha
}  // namespace peagle
