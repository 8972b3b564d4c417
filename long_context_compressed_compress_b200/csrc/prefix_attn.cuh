// Arguments shared by the two kernels of hca_prefix_attn_fwd.
#pragma once

#include "common.cuh"

namespace csa {

struct PrefixAttnArgs {
  const void* q;
  const void* pool;
  const int32_t* table;
  const int32_t* held;
  const int32_t* group_off;
  const int32_t* group_seq;
  const int32_t* group_shared;
  const void* kv_raw;
  const float* sink;
  const int32_t* q_pos0;
  void* out;
  float* lse;
  int* status;
  float tau;
  int N, P, max_pages, G, n_seq, W, B, T, H, m, raw_cap;
};

// Entries of sequence b that position p sees and the sequence's pages hold.
__device__ __forceinline__ int visible_entries(const PrefixAttnArgs& a, int b, long long p) {
  if (p < 0) return 0;
  const uint32_t cap = static_cast<uint32_t>(max(min(a.held[b], a.max_pages), 0)) * a.P;      // below 2^31
  return static_cast<int>(min(static_cast<uint32_t>(p + 1) / static_cast<uint32_t>(a.m), cap));
}

int launch_prefix_attn_simt(const PrefixAttnArgs& a, int D, int dtype, cudaStream_t st);
int launch_prefix_attn_tc(const PrefixAttnArgs& a, cudaStream_t st);   // bf16, D = 128, H <= 128

}  // namespace csa
