// hca_prefix_attn_fwd on CUDA cores, in fp32: the fp32 types (the tensor cores
// have no fp32 kind) and the bf16 shapes that the tcgen05 kernel does not take.
//
//   l_j = tau <q, k_j>;  out = sum_j e^{l_j} k_j / (e^sigma + sum_j e^{l_j})
//
// A cluster shares one query token and 8 of its heads; warp = one head.  Keys come in
// tiles of 32 (visible entries at multiples of 32, then the window, newest
// first), tile i to rank i % c, as fp32 in shared memory: a lane forms the logit of
// one key (its row in 16-byte reads, rows 4 floats apart from a multiple of the
// banks), the warp joins the running maximum and sum, then a lane sums D / 32 dims
// over the keys.  The next tile's loads are under way meanwhile.  The ranks'
// (O, M, l) join in distributed shared memory, in rank order.  c depends on the
// cache's capacity alone, so a row's bits do not depend on batch or grouping.
//
// Bound by latency at the sizes of decoding (a tile is some 300 instructions a
// warp, a short call three tiles a rank) and by fp32 FMAs at long ones.
#include "common.cuh"
#include "prefix_attn.cuh"

namespace csa {
namespace {

constexpr int kHeads = 8;
constexpr int kKeys = 32;
constexpr int kMost = 8;         // ranks

__device__ __forceinline__ float peer_f(const float* p, int rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kHeads) prefix_attn_simt_kernel(const PrefixAttnArgs a, int c) {
  constexpr int DL = D / 32, LD = D + 4;
  constexpr int VEC = 16 / sizeof(T), CH = D / VEC;                // values, vectors a row
  constexpr int NV = kKeys * CH / (32 * kHeads);                   // vectors a thread
  static_assert(kKeys * CH % (32 * kHeads) == 0, "");
  __shared__ __align__(16) float keys[2][kKeys][LD];
  __shared__ __align__(16) float qs[kHeads][D];
  __shared__ const T* rowptr[2][kKeys];
  __shared__ float o_part[kHeads][D], m_part[kHeads], l_part[kHeads];

  const int hgroups = (a.H + kHeads - 1) / kHeads;
  const int unit = blockIdx.x / c, rank = blockIdx.x - unit * c;
  const int hg = unit % hgroups, pair = unit / hgroups;
  const int b = a.group_seq[pair / a.T], t = pair % a.T;
  if (b < 0 || b >= a.B) {                      // (the whole cluster leaves)
    if (threadIdx.x == 0) atomicCAS(a.status, 0, CSA_ERR_INVALID_ARG | (4 << 8));
    return;
  }
  const long long p = static_cast<long long>(a.q_pos0[b]) + t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = hg * kHeads + warp;
  const size_t row0 = (static_cast<size_t>(b) * a.T + t) * a.H;
  for (int e = threadIdx.x; e < kHeads * D; e += 32 * kHeads) {
    const int hh = hg * kHeads + e / D;
    qs[e / D][e % D] = hh < a.H ? to_f(static_cast<const T*>(a.q)[(row0 + hh) * D + e % D]) * a.tau : 0.f;
  }
  const int n_ent = visible_entries(a, b, p);
  const int n_win = p < 0 ? 0 : static_cast<int>(min(static_cast<long long>(a.W), p + 1));
  const int ent_tiles = (n_ent + kKeys - 1) / kKeys, win_tiles = (n_win + kKeys - 1) / kKeys;
  // this rank's tiles: entries rank, rank + c, ..; window tiles likewise
  const int my_ent = ent_tiles > rank ? (ent_tiles - rank + c - 1) / c : 0;
  const int my_all = my_ent + (win_tiles > rank ? (win_tiles - rank + c - 1) / c : 0);
  const int32_t* tab = a.table + static_cast<size_t>(b) * a.max_pages;

  // Where key x of tile i lies (null: not there).
  auto find = [&](int i, int x) -> const T* {
    if (i < my_ent) {
      const int s = (rank + i * c) * kKeys + x;
      if (s >= n_ent) return nullptr;
      const int id = tab[s / a.P];
      if (id < 0 || id >= a.N) return nullptr;
      return static_cast<const T*>(a.pool) + (static_cast<size_t>(id) * a.P + s % a.P) * D;
    }
    if (i >= my_all) return nullptr;
    const int back = (rank + (i - my_ent) * c) * kKeys + x;
    if (back >= n_win) return nullptr;
    return static_cast<const T*>(a.kv_raw) +
           (static_cast<size_t>(b) * a.raw_cap + static_cast<size_t>((p - back) % a.raw_cap)) * D;
  };
  uint4 raw[NV];
  auto fetch = [&](int i) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = threadIdx.x + k * 32 * kHeads;
      const T* r = rowptr[i & 1][e / CH];
      raw[k] = r ? *reinterpret_cast<const uint4*>(r + (e % CH) * VEC) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  auto stage = [&](int i) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = threadIdx.x + k * 32 * kHeads;
      const T* v = reinterpret_cast<const T*>(&raw[k]);
#pragma unroll
      for (int j = 0; j < VEC; j += 4)
        *reinterpret_cast<float4*>(&keys[i & 1][e / CH][(e % CH) * VEC + j]) =
            make_float4(to_f(v[j]), to_f(v[j + 1]), to_f(v[j + 2]), to_f(v[j + 3]));
    }
  };

  float acc[DL], mrun = -INFINITY, lsum = 0.f;
#pragma unroll
  for (int i = 0; i < DL; ++i) acc[i] = 0.f;
  if (threadIdx.x < 2 * kKeys) rowptr[threadIdx.x / kKeys][threadIdx.x % kKeys] = find(threadIdx.x / kKeys, threadIdx.x % kKeys);
  __syncthreads();
  if (my_all > 0) {
    fetch(0);
    stage(0);
  }
  __syncthreads();
  for (int i = 0; i < my_all; ++i) {
    if (i + 1 < my_all) fetch(i + 1);
    // (a lane's own key, before the slot is given to tile i + 2)
    const bool there = rowptr[i & 1][lane] != nullptr;
    float x = 0.f;
    {
      const float4* kr = reinterpret_cast<const float4*>(keys[i & 1][lane]);
      const float4* qr = reinterpret_cast<const float4*>(qs[warp]);
      float x4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int d = 0; d < D / 4; ++d) {
        const float4 kv = kr[d], qv = qr[d];
        x4[0] = fmaf(kv.x, qv.x, x4[0]);
        x4[1] = fmaf(kv.y, qv.y, x4[1]);
        x4[2] = fmaf(kv.z, qv.z, x4[2]);
        x4[3] = fmaf(kv.w, qv.w, x4[3]);
      }
      x = (x4[0] + x4[1]) + (x4[2] + x4[3]);
    }
    float mx = there ? x : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(mrun, mx), base = mn == -INFINITY ? 0.f : mn;
    const float f = mrun == -INFINITY ? 0.f : expf(mrun - base);
    const float w = there ? expf(x - base) : 0.f;
    float ws = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
    lsum = fmaf(lsum, f, ws);
    mrun = mn;
#pragma unroll
    for (int d = 0; d < DL; ++d) acc[d] *= f;
    const uint32_t present = __ballot_sync(0xffffffffu, there);
    const int last = present ? 32 - __clz(present) : 0;
#pragma unroll 8
    for (int k = 0; k < last; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
#pragma unroll
      for (int d = 0; d < DL; ++d) acc[d] = fmaf(wk, keys[i & 1][k][lane + 32 * d], acc[d]);
    }
    __syncthreads();                             // tile i's keys and pointers are read
    if (i + 1 < my_all) stage(i + 1);
    if (threadIdx.x < kKeys) rowptr[i & 1][threadIdx.x] = find(i + 2, threadIdx.x);
    __syncthreads();
  }

  // the ranks' parts, joined by the rank that owns the head
#pragma unroll
  for (int d = 0; d < DL; ++d) o_part[warp][lane + 32 * d] = acc[d];
  if (lane == 0) { m_part[warp] = mrun; l_part[warp] = lsum; }
  cluster_sync();
  if (warp % c == rank && h < a.H) {
    float mk[kMost], M = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMost; ++k)
      if (k < c) { mk[k] = peer_f(&m_part[warp], k); M = fmaxf(M, mk[k]); }
    float L = 0.f, res[DL];
#pragma unroll
    for (int d = 0; d < DL; ++d) res[d] = 0.f;
#pragma unroll
    for (int k = 0; k < kMost; ++k)
      if (k < c) {
        // (M is not NaN; a NaN logit is in l and O)
        const float f = mk[k] == -INFINITY ? (M == -INFINITY ? 1.f : 0.f) : expf(mk[k] - M);
        L = fmaf(f, peer_f(&l_part[warp], k), L);
#pragma unroll
        for (int d = 0; d < DL; ++d) res[d] = fmaf(f, peer_f(&o_part[warp][lane + 32 * d], k), res[d]);
      }
    float scale = 0.f;
    if (L != 0.f) {
      const float sg = a.sink ? a.sink[h] : -INFINITY;
      const float X = fmaxf(M, sg), f = X == -INFINITY ? 1.f : expf(M - X);
      scale = __fdiv_rn(f, fmaf(L, f, X == -INFINITY ? 0.f : expf(sg - X)));
    }
    T* out = static_cast<T*>(a.out) + (row0 + h) * D;
#pragma unroll
    for (int d = 0; d < DL; ++d) out[lane + 32 * d] = static_cast<T>(res[d] * scale);
    if (a.lse && lane == 0) a.lse[row0 + h] = L == 0.f ? -INFINITY : M + logf(L);
  }
  cluster_sync();                                // peers have read this CTA's parts
}

template <typename T, int D>
int launch(const PrefixAttnArgs& a, cudaStream_t st) {
  // ranks for the longest sequence that the cache can hold, two tiles each at least
  const long long tiles = (static_cast<long long>(a.max_pages) * a.P + kKeys - 1) / kKeys;
  int c = 1;
  while (c < kMost && 2 * c <= tiles) c *= 2;
  const long long grid = static_cast<long long>(a.n_seq) * a.T * ((a.H + kHeads - 1) / kHeads) * c;
  CSA_REQUIRE(grid < (1ll << 31), CSA_ERR_UNSUPPORTED);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(32 * kHeads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, prefix_attn_simt_kernel<T, D>, a, c);
  if (e != cudaSuccess) return set_cuda_error(e);
  return check_launch();
}

}  // namespace

int launch_prefix_attn_simt(const PrefixAttnArgs& a, int D, int dtype, cudaStream_t st) {
  if (dtype == CSA_F32) return D == 64 ? launch<float, 64>(a, st) : launch<float, 128>(a, st);
  return D == 64 ? launch<__nv_bfloat16, 64>(a, st) : launch<__nv_bfloat16, 128>(a, st);
}

}  // namespace csa
