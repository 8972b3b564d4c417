// Entry point of hca_prefix_attn_fwd: argument checks and the choice of kernel.
#include "prefix_attn.cuh"

using namespace csa;

extern "C" int hca_prefix_attn_fwd(const void* q, const void* pool, int N, int P, const int32_t* table,
                                   const int32_t* held, int max_pages, const int32_t* group_off,
                                   const int32_t* group_seq, const int32_t* group_shared, int G, int n_seq,
                                   const void* kv_raw, const float* sink, float tau, int W, int B, int T, int H, int D,
                                   int m, int raw_cap, const int32_t* q_pos0, void* out, float* lse, int dtype,
                                   int32_t* status, csa_stream_t stream) {
  CSA_REQUIRE(q && pool && table && held && group_off && q_pos0 && out, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(G >= 0 && n_seq >= 0 && (n_seq == 0 || (group_seq && group_shared)), CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(N >= 0 && P >= 1 && max_pages >= 1 && m >= 1, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(B >= 0 && T >= 0 && H >= 0 && W >= 0, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(W == 0 || (kv_raw && raw_cap >= 1 && static_cast<long long>(raw_cap) >= static_cast<long long>(W) + T - 1),
              CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(dtype == CSA_F32 || dtype == CSA_BF16, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE((D == 64 || D == 128) && H <= 1024, CSA_ERR_UNSUPPORTED);
  CSA_REQUIRE(static_cast<long long>(max_pages) * P < (1ll << 31), CSA_ERR_UNSUPPORTED);
  CSA_REQUIRE(aligned16(q) && aligned16(pool) && aligned16(kv_raw) && aligned16(out), CSA_ERR_ALIGNMENT);
  if (n_seq == 0 || G == 0 || T == 0 || H == 0 || B == 0) return CSA_OK;
  PrefixAttnArgs a;
  a.q = q; a.pool = pool; a.table = table; a.held = held; a.group_off = group_off; a.group_seq = group_seq;
  a.group_shared = group_shared; a.kv_raw = kv_raw; a.sink = sink; a.q_pos0 = q_pos0; a.out = out; a.lse = lse;
  a.status = status_word(status);
  CSA_REQUIRE(a.status != nullptr, CSA_ERR_CUDA);
  a.tau = tau; a.N = N; a.P = P; a.max_pages = max_pages; a.G = G; a.n_seq = n_seq; a.W = W; a.B = B; a.T = T;
  a.H = H; a.m = m; a.raw_cap = raw_cap;
  if (dtype == CSA_BF16 && D == 128 && H <= 128) return launch_prefix_attn_tc(a, reinterpret_cast<cudaStream_t>(stream));
  return launch_prefix_attn_simt(a, D, dtype, reinterpret_cast<cudaStream_t>(stream));
}
