// hca_prefix_attn_fwd on CUDA cores, in fp32: the fp32 types (the tensor cores
// have no fp32 kind) and the bf16 shapes that the tcgen05 kernel does not take.
//
// CTA = (query token, 8 heads); warp = one head; lane = D / 32 dims of q and of
// the running output.  Keys are the visible paged entries, then the window rows,
// staged 64 at a time in shared memory as fp32; the softmax is the online form
// with a running maximum and sum.
#include "common.cuh"
#include "prefix_attn.cuh"

namespace csa {

constexpr int kPsHeads = 8;
constexpr int kPsKeys = 64;

template <typename T, int D>
__global__ void __launch_bounds__(256) prefix_attn_simt_kernel(const PrefixAttnArgs a) {
  constexpr int DL = D / 32;
  __shared__ float keys[kPsKeys][D];
  __shared__ const T* rowptr[kPsKeys];
  const int ngroups = (a.H + kPsHeads - 1) / kPsHeads;
  const int hg = blockIdx.x % ngroups;
  const int pair = blockIdx.x / ngroups;
  const int b = a.group_seq[pair / a.T], t = pair % a.T;
  if (b < 0 || b >= a.B) {
    if (threadIdx.x == 0) atomicCAS(a.status, 0, CSA_ERR_INVALID_ARG | (4 << 8));
    return;
  }
  const long long p = static_cast<long long>(a.q_pos0[b]) + t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = hg * kPsHeads + warp;
  const bool hok = h < a.H;
  const size_t row = (static_cast<size_t>(b) * a.T + t) * a.H + (hok ? h : 0);
  const T* q = static_cast<const T*>(a.q) + row * D;
  float qv[DL], acc[DL];
#pragma unroll
  for (int i = 0; i < DL; ++i) { qv[i] = to_f(q[lane + 32 * i]) * a.tau; acc[i] = 0.f; }
  float mrun = -INFINITY, lsum = 0.f;
  const int n_ent = visible_entries(a, b, p);
  const int n_win = p < 0 ? 0 : static_cast<int>(min(static_cast<long long>(a.W), p + 1));
  const int n_all = n_ent + n_win;
  const int32_t* tab = a.table + static_cast<size_t>(b) * a.max_pages;
  for (int base = 0; base < n_all; base += kPsKeys) {
    const int cnt = min(kPsKeys, n_all - base);
    __syncthreads();
    if (threadIdx.x < cnt) {
      const int j = base + threadIdx.x;
      const T* ptr = nullptr;
      if (j < n_ent) {
        const int id = tab[j / a.P];
        if (id >= 0 && id < a.N) ptr = static_cast<const T*>(a.pool) + (static_cast<size_t>(id) * a.P + j % a.P) * D;
      } else {
        const long long tok = p - (j - n_ent);
        ptr = static_cast<const T*>(a.kv_raw) + (static_cast<size_t>(b) * a.raw_cap + static_cast<size_t>(tok % a.raw_cap)) * D;
      }
      rowptr[threadIdx.x] = ptr;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < cnt * D; e += blockDim.x) {
      const int kk = e / D, d = e - kk * D;
      const T* ptr = rowptr[kk];
      keys[kk][d] = ptr ? to_f(ptr[d]) : 0.f;
    }
    __syncthreads();
    if (!hok) continue;
    for (int kk = 0; kk < cnt; ++kk) {
      if (rowptr[kk] == nullptr) continue;
      float l = 0.f;
#pragma unroll
      for (int i = 0; i < DL; ++i) l = fmaf(qv[i], keys[kk][lane + 32 * i], l);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (l > mrun) {
        const float sc = expf(mrun - l);
        lsum *= sc;
#pragma unroll
        for (int i = 0; i < DL; ++i) acc[i] *= sc;
        mrun = l;
      }
      const float pe = expf(l - mrun);
      lsum += pe;
#pragma unroll
      for (int i = 0; i < DL; ++i) acc[i] = fmaf(pe, keys[kk][lane + 32 * i], acc[i]);
    }
  }
  if (!hok) return;
  const float sg = a.sink ? a.sink[h] : -INFINITY;
  // a stabiliser that only the sink sets must not make 0 * inf of an empty row
  float scale = 0.f;
  if (lsum != 0.f) {
    const float M = fmaxf(mrun, sg);
    const float f = expf(mrun - M);
    scale = __fdiv_rn(f, fmaf(lsum, f, expf(sg - M)));
  }
  T* out = static_cast<T*>(a.out) + row * D;
#pragma unroll
  for (int i = 0; i < DL; ++i) out[lane + 32 * i] = static_cast<T>(acc[i] * scale);
  if (a.lse && lane == 0) a.lse[row] = lsum == 0.f ? -INFINITY : mrun + logf(lsum);
}

int launch_prefix_attn_simt(const PrefixAttnArgs& a, int D, int dtype, cudaStream_t st) {
  const long long grid = static_cast<long long>(a.n_seq) * a.T * ((a.H + kPsHeads - 1) / kPsHeads);
  CSA_REQUIRE(grid < (1ll << 31), CSA_ERR_UNSUPPORTED);
#define PS(TT, DD) prefix_attn_simt_kernel<TT, DD><<<static_cast<unsigned>(grid), 256, 0, st>>>(a)
  if (dtype == CSA_F32) {
    if (D == 64) PS(float, 64); else PS(float, 128);
  } else {
    if (D == 64) PS(__nv_bfloat16, 64); else PS(__nv_bfloat16, 128);
  }
#undef PS
  return check_launch();
}

}  // namespace csa
