// hca_paged_append: the m:1 gated pooling of new tokens into paged entries, from
// one decode token to a whole prompt, with the open block carried in fp32.
//
// For each channel a set of tokens is summed up by (M, Z, A) = (max z,
// sum e^{z-M}, sum e^{z-M} a); two sets join by rescaling to the larger M, and the
// entry is A / Z.  The order of the joins is fixed by positions alone: the 16
// tokens of a run one after the other, then the block's runs in ascending
// order.  So a token sequence gives the same bits however calls split it, and the
// runs of a block are summed in parallel.
//
// Bound by HBM: a and z are read once.  D / 8 lanes hold a row (16-byte loads of
// bf16) and a thread walks the 16 tokens of one run, all of whose loads are
// independent of its arithmetic.
#include <cfloat>

#include "rope.cuh"

namespace csa {

constexpr int kRun = 16;     // tokens per run
constexpr int kSlots = 8;    // runs (of one or more blocks) a CTA sums at once

struct AppendArgs {
  const void* a;
  const void* z;
  const int32_t* pos0;
  const int32_t* lens;
  const float* carry_in;
  float* carry_out;
  void* pool;
  const int32_t* table;
  const int32_t* held;
  const float* weight;
  const double* inv_freq;
  int* status;
  float eps;
  int T, m, N, P, max_pages, R, flags;
  int runs;          // per block
  int sg;            // slots per block
  int ctas_seq;      // CTAs per sequence: one for its first and last blocks, the rest for those between
};

struct State8 {
  float M[8], Z[8], A[8];
};
__device__ __forceinline__ void empty_state(State8& s) {
#pragma unroll
  for (int c = 0; c < 8; ++c) { s.M[c] = -FLT_MAX; s.Z[c] = 0.f; s.A[c] = 0.f; }
}
// One more token.  A gate of -inf has weight 0; the larger of M and z keeps weight 1,
// so one exponential serves both.
__device__ __forceinline__ void add_token(float& M, float& Z, float& A, float z, float a) {
  const float d = z - M;
  const float e = expf(-fabsf(d));
  const bool up = d > 0.f;
  const float keep = up ? e : 1.f, w = up ? 1.f : e;
  Z = fmaf(Z, keep, w);
  // a dropped token's value (weight 0) is not looked at
  A = fmaf(A, keep, w > 0.f ? w * a : (w == 0.f ? 0.f : w));
  M = up ? z : M;
}
__device__ __forceinline__ void join(float& M, float& Z, float& A, float m2, float z2, float a2) {
  const float mx = fmaxf(M, m2);
  const float e1 = expf(M - mx), e2 = expf(m2 - mx);
  Z = fmaf(Z, e1, z2 * e2);
  A = fmaf(A, e1, a2 * e2);
  M = mx;
}

template <typename T_, int D>
__global__ void __launch_bounds__(kSlots * D / 8) append_kernel(const AppendArgs a) {
  constexpr int G = D / 8;
  __shared__ float part[kSlots][3][D];
  __shared__ float entry[kSlots][D];
  __shared__ float2 cs[kSlots][D / 2];
  const int b = blockIdx.x / a.ctas_seq, job = blockIdx.x - b * a.ctas_seq;
  const int slot = threadIdx.x / G, l = threadIdx.x % G;   // loading: a run's slot, 8 channels
  const int ch = threadIdx.x;                              // folding: one channel
  const long long p0 = a.pos0[b];
  const int len = p0 < 0 ? 0 : (a.lens ? min(max(a.lens[b], 0), a.T) : a.T);
  const float* cin = a.carry_in + static_cast<size_t>(b) * 6 * D;
  float* cout = a.carry_out + static_cast<size_t>(b) * 6 * D;
  if (len == 0) {
    if (job == 0 && cin != cout)
      for (int i = 0; i < 6; ++i) cout[i * D + ch] = cin[i * D + ch];
    return;
  }
  const long long end = p0 + len;
  const long long first = p0 / a.m, last = end / a.m;   // the open blocks before and after
  const int E = kSlots / a.sg;
  const T_* za = static_cast<const T_*>(a.z) + static_cast<size_t>(b) * a.T * D;
  const T_* aa = static_cast<const T_*>(a.a) + static_cast<size_t>(b) * a.T * D;

  // Passes of this CTA: job 0 takes the first block, then the last (the carry
  // goes in and out through one CTA, so carry_out may be carry_in); job k > 0
  // takes E of the blocks strictly between them.
  const int passes = job == 0 ? (last > first ? 2 : 1) : 1;
  for (int pass = 0; pass < passes; ++pass) {
    const long long blk0 = job == 0 ? (pass == 0 ? first : last) : first + 1 + static_cast<long long>(job - 1) * E;
    const int nblk = job == 0 ? 1 : static_cast<int>(min(static_cast<long long>(E), last - blk0));
    if (nblk <= 0) return;
    const int e = slot / a.sg;
    const bool carried = job == 0 && pass == 0 && p0 % a.m != 0;
    const long long blk = blk0 + e;
    // fold state of this thread's channel, one per block of the CTA
    float M[kSlots], Z[kSlots], A[kSlots];
    float M1 = -FLT_MAX, Z1 = 0.f, A1 = 0.f;   // the run in progress at the end (job 0)
#pragma unroll
    for (int i = 0; i < kSlots; ++i) { M[i] = -FLT_MAX; Z[i] = 0.f; A[i] = 0.f; }
    if (carried) { M[0] = cin[ch]; Z[0] = cin[D + ch]; A[0] = cin[2 * D + ch]; }
    const long long bend = min((blk0 + 1) * a.m, end);   // job 0: where the block's tokens stop
    for (int s0 = 0; s0 < a.runs; s0 += a.sg) {
      const int run = s0 + slot % a.sg;
      State8 st;
      empty_state(st);
      if (e < nblk && run < a.runs) {
        const long long lo = blk * a.m + run * kRun;
        const long long hi = min(lo + kRun, (blk + 1) * a.m);
        if (carried && lo <= p0 && p0 < hi && p0 > lo) {
          Vec8<float>::load(cin + 3 * D + l * 8, st.M);
          Vec8<float>::load(cin + 4 * D + l * 8, st.Z);
          Vec8<float>::load(cin + 5 * D + l * 8, st.A);
        }
        const int t0 = static_cast<int>(max(lo, p0) - p0), t1 = static_cast<int>(min(hi, end) - p0);
#pragma unroll 4
        for (int t = t0; t < t1; ++t) {
          float z8[8], a8[8];
          Vec8<T_>::load(za + static_cast<size_t>(t) * D + l * 8, z8);
          Vec8<T_>::load(aa + static_cast<size_t>(t) * D + l * 8, a8);
#pragma unroll
          for (int c = 0; c < 8; ++c) add_token(st.M[c], st.Z[c], st.A[c], z8[c], a8[c]);
        }
      }
      Vec8<float>::store(&part[slot][0][l * 8], st.M);
      Vec8<float>::store(&part[slot][1][l * 8], st.Z);
      Vec8<float>::store(&part[slot][2][l * 8], st.A);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        if (k >= nblk) break;
        for (int r = 0; r < a.sg && s0 + r < a.runs; ++r) {
          const int i = k * a.sg + r;
          const long long lo = (blk0 + k) * a.m + (s0 + r) * kRun;
          const long long hi = min(lo + kRun, (blk0 + k + 1) * a.m);
          // job 0: a run that ends behind the tokens is still in progress
          if (job == 0 && hi > bend) {
            if (lo < bend) { M1 = part[i][0][ch]; Z1 = part[i][1][ch]; A1 = part[i][2][ch]; }
            continue;
          }
          if (carried && hi <= p0) continue;   // in the carry's first part already
          join(M[k], Z[k], A[k], part[i][0][ch], part[i][1][ch], part[i][2][ch]);
        }
      }
      __syncthreads();
    }
    const bool complete = job != 0 || (pass == 0 && last > first);
    if (!complete) {
      cout[ch] = M[0]; cout[D + ch] = Z[0]; cout[2 * D + ch] = A[0];
      cout[3 * D + ch] = M1; cout[4 * D + ch] = Z1; cout[5 * D + ch] = A1;
      return;
    }
#pragma unroll
    for (int k = 0; k < kSlots; ++k)
      if (k < nblk) entry[k][ch] = Z[k] == 0.f ? 0.f : __fdiv_rn(A[k], Z[k]);
    for (int i = threadIdx.x; i < nblk * (a.R / 2); i += blockDim.x) {
      const int k = i / (a.R / 2), f = i - k * (a.R / 2);
      cs[k][f] = cos_sin_at((blk0 + k) * a.m, a.inv_freq[f], a.flags & CSA_ROPE_INVERSE);
    }
    __syncthreads();
    // slot k finishes entry k
    float v[8];
    Vec8<float>::load(&entry[slot][l * 8], v);
    if (slot >= nblk) {
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = 0.f;
    }
    if (a.flags & CSA_NORM) {
      const float sc = row_rms_scale<D>(v, a.eps);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = v[c] * sc * (a.weight ? a.weight[l * 8 + c] : 1.f);
    }
    LaneRope lr;
    load_lane_rope<D>(lr, cs[slot < nblk ? slot : 0], a.R, a.flags & CSA_ROPE_HALF, l);
    rotate8(v, lr, a.R, a.flags & CSA_ROPE_HALF);
    if (slot < nblk) {
      const long long s = blk0 + slot;
      const long long pi = s / a.P;
      const int hp = min(a.held[b], a.max_pages);
      const int id = pi < hp ? a.table[static_cast<size_t>(b) * a.max_pages + pi] : -1;
      if (id >= 0 && id < a.N)
        Vec8<T_>::store(static_cast<T_*>(a.pool) + (static_cast<size_t>(id) * a.P + s % a.P) * D + l * 8, v);
      else if (l == 0)
        atomicCAS(a.status, 0, CSA_ERR_NO_SPACE | (1 << 8));
    }
    __syncthreads();
  }
}

}  // namespace csa

using namespace csa;

extern "C" int hca_paged_append(const void* a, const void* z, int dtype, int B, int T, int D, int m,
                                const int32_t* pos0, const int32_t* lens, const float* carry_in, float* carry_out,
                                void* pool, int N, int P, const int32_t* table, const int32_t* held, int max_pages,
                                const float* weight, float eps, const double* inv_freq, int R, int flags,
                                int32_t* status, csa_stream_t stream) {
  CSA_REQUIRE(a && z && pos0 && carry_in && carry_out && pool && table && held, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(B >= 0 && T >= 0 && m >= 1 && N >= 0 && P >= 1 && max_pages >= 1, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(R >= 0 && R <= D && (R == 0 || inv_freq) && eps >= 0.f, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE((flags & ~(CSA_NORM | CSA_ROPE_INVERSE | CSA_ROPE_HALF)) == 0, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(dtype == CSA_F32 || dtype == CSA_BF16, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE((D == 64 || D == 128 || D == 256) && R % 16 == 0, CSA_ERR_UNSUPPORTED);
  CSA_REQUIRE(aligned16(a) && aligned16(z) && aligned16(pool) && aligned16(carry_in) && aligned16(carry_out) &&
                  aligned16(weight),
              CSA_ERR_ALIGNMENT);
  // the carry is updated in place or apart, never half over itself
  const ptrdiff_t apart = carry_out - carry_in, cn = static_cast<ptrdiff_t>(B) * 6 * D;
  CSA_REQUIRE(apart == 0 || apart >= cn || -apart >= cn, CSA_ERR_INVALID_ARG);
  if (B == 0) return CSA_OK;
  AppendArgs g;
  g.a = a; g.z = z; g.pos0 = pos0; g.lens = lens; g.carry_in = carry_in; g.carry_out = carry_out; g.pool = pool;
  g.table = table; g.held = held; g.weight = weight; g.inv_freq = inv_freq; g.eps = eps;
  g.T = T; g.m = m; g.N = N; g.P = P; g.max_pages = max_pages; g.R = R; g.flags = flags;
  g.status = status_word(status);
  CSA_REQUIRE(g.status != nullptr, CSA_ERR_CUDA);
  g.runs = (m + kRun - 1) / kRun;
  // slots per block: a power of two, so that kSlots / sg blocks fit a CTA
  g.sg = 1;
  while (g.sg < kSlots && g.sg < g.runs) g.sg *= 2;
  const int E = kSlots / g.sg;
  g.ctas_seq = 1 + (T / m + E - 1) / E;
  const long long grid = static_cast<long long>(B) * g.ctas_seq;
  CSA_REQUIRE(grid < (1ll << 31), CSA_ERR_UNSUPPORTED);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
#define AP(TT, DD) append_kernel<TT, DD><<<static_cast<unsigned>(grid), kSlots * DD / 8, 0, st>>>(g)
  if (dtype == CSA_F32) {
    if (D == 64) AP(float, 64); else if (D == 128) AP(float, 128); else AP(float, 256);
  } else {
    if (D == 64) AP(__nv_bfloat16, 64); else if (D == 128) AP(__nv_bfloat16, 128); else AP(__nv_bfloat16, 256);
  }
#undef AP
  return check_launch();
}
