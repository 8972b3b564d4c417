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
// Bound by HBM: a and z are read once.  D / 4 lanes hold a row and a thread walks the
// 16 tokens of one run, two tokens of loads ahead of its arithmetic (2 x 128K tokens
// of 128 channels: 4.8 TB/s, against 6.6 for a copy, with half of the issue slots in
// use; 72 registers a thread let 28 warps share an SM, whose loads do not cover all of
// their latency).
#include <cfloat>

#include "rope.cuh"

namespace csa {

constexpr int kRun = 16;     // tokens per run
// Runs (of one or more blocks) a CTA sums at once, and threads an SM holds at least: small
// CTAs, whose sums and joins overlap each other's (for 2 x 128K tokens 34.1 us with
// 8 runs, 27.4 us with 4; 640, 768 or 1024 threads an SM: 30.3, 30.6, 31.0 us).  Blocks of
// one run, of which a CTA takes four (2 x 128K tokens, m = 4: 62.5 us, 65 with 896
// threads, 78 with 640; 81 with a token's loads at a time and sums through shared memory).
constexpr int kSlots = 4;
constexpr int kSmThreads = 896, kSmThreadsOne = 768;

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
  int ctas_seq;      // CTAs per sequence: one for its first and last blocks, the rest for those between
};

// Exponentials are 2^(x log2 e) on the special-function unit: 2^-22 of the result, and |x|
// times three half steps of fp32 (x itself, the constant, the product).  For a block of n
// tokens, u of which raise the maximum, with gates within d of it, Z and A are off by less
// than (n + 4 u + 3 d + 5 n / 16 + 8) 2^-24 of their terms' magnitude, most of it the n
// roundings of a sum in any order.  (Weights below 2^-126 become 0.)
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// A thread sums 4 channels: 8 would need twice the registers that let 768 threads
// share an SM.
struct State4 {
  float M[4], Z[4], A[4];
};
__device__ __forceinline__ void empty_state(State4& s) {
#pragma unroll
  for (int c = 0; c < 4; ++c) { s.M[c] = -FLT_MAX; s.Z[c] = 0.f; s.A[c] = 0.f; }
}
__device__ __forceinline__ void load4(const float* p, float v[4]) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
// 4 values as loaded (read once: they bypass L1).
template <typename T> struct Raw4;
template <> struct Raw4<float> {
  float4 x;
  __device__ __forceinline__ void load(const float* p) { x = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void get(float v[4]) const { v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; }
};
template <> struct Raw4<__nv_bfloat16> {
  uint2 x;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = __ldcs(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void get(float v[4]) const {
    v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xffff0000u);
    v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xffff0000u);
  }
};
__device__ __forceinline__ void store4(float* p, const float v[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
// (d0, d1) = (a0, a1) * (b0, b1) + (c0, c1) on the packed fp32 pipe
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// One more token, two channels.  The larger of M and z keeps weight 1, so one
// exponential serves both.  A gate of -inf has weight 0; what its token's value
// may then do to A (0 * inf) is seen to once a run, by the careful form, which does
// not look at it.
template <bool CAREFUL>
__device__ __forceinline__ void add_token2(float* M, float* Z, float* A, const float* z, const float* a) {
  float d[2], keep[2], w[2], wa[2];
  fma2(d[0], d[1], M[0], M[1], -1.f, -1.f, z[0], z[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float e = exp2_fast(fabsf(d[i]) * -kLog2e);
    const bool up = d[i] > 0.f;
    keep[i] = up ? e : 1.f;
    w[i] = up ? 1.f : e;
    M[i] = up ? z[i] : M[i];
  }
  fma2(Z[0], Z[1], Z[0], Z[1], keep[0], keep[1], w[0], w[1]);
  mul2(wa[0], wa[1], w[0], w[1], a[0], a[1]);
  if (CAREFUL) {
    wa[0] = w[0] == 0.f ? 0.f : wa[0];
    wa[1] = w[1] == 0.f ? 0.f : wa[1];
  }
  fma2(A[0], A[1], A[0], A[1], keep[0], keep[1], wa[0], wa[1]);
}
__device__ __forceinline__ void join(float& M, float& Z, float& A, float m2, float z2, float a2) {
  const float mx = fmaxf(M, m2);
  const float e1 = exp2_fast((M - mx) * kLog2e), e2 = exp2_fast((m2 - mx) * kLog2e);
  Z = fmaf(Z, e1, z2 * e2);
  A = fmaf(A, e1, a2 * e2);
  M = mx;
}

// Part of a run, kBatch tokens of loads at a time.
template <typename T_, int D, bool CAREFUL, int kBatch>
__device__ __forceinline__ void add_tokens(State4& st, const T_* z, const T_* a, int t0, int t1) {
#pragma unroll 1
  for (int t = t0; t < t1; t += kBatch) {
    Raw4<T_> zr[kBatch], ar[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (t + i < t1) {
        zr[i].load(z + static_cast<size_t>(t + i) * D);
        ar[i].load(a + static_cast<size_t>(t + i) * D);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (t + i >= t1) break;
      float z4[4], a4[4];
      zr[i].get(z4);
      ar[i].get(a4);
#pragma unroll
      for (int c = 0; c < 4; c += 2) add_token2<CAREFUL>(st.M + c, st.Z + c, st.A + c, z4 + c, a4 + c);
    }
  }
}
// A whole run: the next kAhead tokens are on their way while these are added.
constexpr int kAhead = 2;
template <typename T_, int D>
__device__ __forceinline__ void add_run(State4& st, const T_* z, const T_* a) {
  Raw4<T_> zr[2][kAhead], ar[2][kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) { zr[0][i].load(z + i * D); ar[0][i].load(a + i * D); }
#pragma unroll
  for (int k = 0; k < kRun / kAhead; ++k) {
    if (k + 1 < kRun / kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        zr[(k + 1) & 1][i].load(z + ((k + 1) * kAhead + i) * D);
        ar[(k + 1) & 1][i].load(a + ((k + 1) * kAhead + i) * D);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float z4[4], a4[4];
      zr[k & 1][i].get(z4);
      ar[k & 1][i].get(a4);
#pragma unroll
      for (int c = 0; c < 4; c += 2) add_token2<false>(st.M + c, st.Z + c, st.A + c, z4 + c, a4 + c);
    }
  }
}

// E blocks a CTA, kSlots / E runs of each at once.
template <typename T_, int D, int E>
__global__ void __launch_bounds__(kSlots * D / 4, (E == kSlots ? kSmThreadsOne : kSmThreads) / (kSlots * D / 4))
    append_kernel(const AppendArgs a) {
  constexpr int G = D / 8, L = D / 4, SG = kSlots / E;
  // Runs a thread sums before they are joined (for 2 x 128K tokens 27.0 us with one).
  constexpr int kTurns = E == 1 ? 2 : 1;
  __shared__ float part[kTurns * kSlots][3][D];
  __shared__ float entry[E][D];
  const int b = blockIdx.x / a.ctas_seq, job = blockIdx.x - b * a.ctas_seq;
  const int slot = threadIdx.x / L, q = threadIdx.x % L;   // summing: a run's slot, 4 channels
  const int ch = threadIdx.x;                              // folding: one channel (below D)
  const int row = threadIdx.x / G, l = threadIdx.x % G;    // finishing: an entry, 8 channels
  const int pos = a.pos0[b];
  const int len = pos < 0 ? 0 : (a.lens ? min(max(a.lens[b], 0), a.T) : a.T);
  const float* cin = a.carry_in + static_cast<size_t>(b) * 6 * D;
  float* cout = a.carry_out + static_cast<size_t>(b) * 6 * D;
  if (len == 0) {
    if (job == 0 && cin != cout && ch < D)
      for (int i = 0; i < 6; ++i) cout[i * D + ch] = cin[i * D + ch];
    return;
  }
  // Positions from here on count from the start of the first block (block `first`):
  // p0 becomes the tokens already in it.
  const int first = static_cast<int>(pos) / a.m, p0 = static_cast<int>(pos) - first * a.m;
  const int end = p0 + len, last = end / a.m;           // tokens, and the open block behind them
  const T_* za = static_cast<const T_*>(a.z) + static_cast<size_t>(b) * a.T * D + q * 4;
  const T_* aa = static_cast<const T_*>(a.a) + static_cast<size_t>(b) * a.T * D + q * 4;

  // Passes of this CTA: job 0 takes the first block, then the last (the carry
  // goes in and out through one CTA, so carry_out may be carry_in); job k > 0
  // takes E of the blocks strictly between them.
  const int passes = job == 0 && last > 0 ? 2 : 1;
  for (int pass = 0; pass < passes; ++pass) {
    const int blk0 = job == 0 ? (pass == 0 ? 0 : last) : 1 + (job - 1) * E;
    const int nblk = job == 0 ? 1 : min(E, last - blk0);
    if (nblk <= 0) return;
    const int e = slot / SG;
    const bool carried = job == 0 && pass == 0 && p0 != 0;
    // fold state of this thread's channel, one per block of the CTA
    float M[E], Z[E], A[E];
    float M1 = -FLT_MAX, Z1 = 0.f, A1 = 0.f;   // the run in progress at the end (job 0)
#pragma unroll
    for (int i = 0; i < E; ++i) { M[i] = -FLT_MAX; Z[i] = 0.f; A[i] = 0.f; }
    if (carried && ch < D) { M[0] = cin[ch]; Z[0] = cin[D + ch]; A[0] = cin[2 * D + ch]; }
    const int bend = min((blk0 + 1) * a.m, end);   // job 0: where the block's tokens stop
    for (int s0 = 0; s0 < a.runs; s0 += kTurns * SG) {
#pragma unroll 1
      for (int turn = 0; turn < kTurns; ++turn) {
        const int run = s0 + turn * SG + slot % SG;
        if (turn > 0 && s0 + turn * SG >= a.runs) break;
        State4 st;
        empty_state(st);
        if (e < nblk && run < a.runs) {
          const int lo = (blk0 + e) * a.m + run * kRun;
          const int hi = min(lo + kRun, (blk0 + e + 1) * a.m);
          const int t0 = max(lo, p0) - p0, t1 = min(hi, end) - p0;
          auto start = [&]() {
            empty_state(st);
            if (carried && lo < p0 && p0 < hi) {
              load4(cin + 3 * D + q * 4, st.M);
              load4(cin + 4 * D + q * 4, st.Z);
              load4(cin + 5 * D + q * 4, st.A);
            }
          };
          start();
          if (t1 - t0 == kRun) add_run<T_, D>(st, za + static_cast<size_t>(t0) * D, aa + static_cast<size_t>(t0) * D);
          else add_tokens<T_, D, false, E == kSlots ? 4 : 1>(st, za, aa, t0, t1);
          bool fine = true;
#pragma unroll
          for (int c = 0; c < 4; ++c) fine = fine && fabsf(st.A[c]) <= FLT_MAX;
          if (!fine) {
            start();
            add_tokens<T_, D, true, 1>(st, za, aa, t0, t1);
          }
        }
        if (E == kSlots && job != 0) {
          // a block is one run: its sums are the entry's
          float v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = st.Z[c] == 0.f ? 0.f : __fdiv_rn(st.A[c], st.Z[c]);
          store4(&entry[slot][q * 4], v);
          break;
        }
        store4(&part[turn * kSlots + slot][0][q * 4], st.M);
        store4(&part[turn * kSlots + slot][1][q * 4], st.Z);
        store4(&part[turn * kSlots + slot][2][q * 4], st.A);
      }
      if (E == kSlots && job != 0) break;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < E; ++k) {
        if (k >= nblk || ch >= D) break;
#pragma unroll
        for (int r = 0; r < kTurns * SG; ++r) {
          if (s0 + r >= a.runs) break;
          const int i = r / SG * kSlots + k * SG + r % SG;
          const int lo = (blk0 + k) * a.m + (s0 + r) * kRun;
          const int hi = min(lo + kRun, (blk0 + k + 1) * a.m);
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
    const bool complete = job != 0 || (pass == 0 && last > 0);
    if (!complete) {
      if (ch >= D) return;
      cout[ch] = M[0]; cout[D + ch] = Z[0]; cout[2 * D + ch] = A[0];
      cout[3 * D + ch] = M1; cout[4 * D + ch] = Z1; cout[5 * D + ch] = A1;
      return;
    }
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (ch < D && !(E == kSlots && job != 0)) entry[k][ch] = Z[k] == 0.f ? 0.f : __fdiv_rn(A[k], Z[k]);
    __syncthreads();
    // row k of lanes finishes entry k (whole warps take part: rows behind the last are zeros)
    if (threadIdx.x < (E * G + 31) / 32 * 32) {
      const bool half = a.flags & CSA_ROPE_HALF;
      const LaneRuns own = lane_runs<D>(l, a.R, half);
      Raw8<float, true> raw;
      float v[8];
      if (row < nblk) raw.load(&entry[row][own.a], own.b - own.a);
      else raw.zero();
      raw.get(v);
      if (a.flags & CSA_NORM) {
        const float sc = row_rms_scale<D>(v, a.eps);
        float w[8];
        weights8(a.weight, own, w);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] *= sc * w[c];
      }
      if (a.R > 0) {
        LaneRope lr;
        const long long at = static_cast<long long>(first + blk0 + min(row, nblk - 1)) * a.m;
        lane_rope_alone<D>(lr, at, a.inv_freq, a.R, a.flags & CSA_ROPE_INVERSE, l);
        if (half) rotate8<true>(v, lr);
        else rotate8<false>(v, lr);
      }
      if (row < nblk) {
        const int s = first + blk0 + row, pi = s / a.P;
        const int hp = min(a.held[b], a.max_pages);
        const int id = pi < hp ? a.table[static_cast<size_t>(b) * a.max_pages + pi] : -1;
        if (id >= 0 && id < a.N)
          store8<true>(static_cast<T_*>(a.pool) + (static_cast<size_t>(id) * a.P + s % a.P) * D + own.a, own.b - own.a, v);
        else if (l == 0)
          atomicCAS(a.status, 0, CSA_ERR_NO_SPACE | (1 << 8));
      }
    }
    __syncthreads();
  }
}

template <typename T_, int D>
int launch_append(const AppendArgs& g, int B, int E, cudaStream_t st) {
  const long long grid = static_cast<long long>(B) * g.ctas_seq;
  CSA_REQUIRE(grid < (1ll << 31), CSA_ERR_UNSUPPORTED);
  const unsigned n = static_cast<unsigned>(grid);
  constexpr int kThreads = kSlots * D / 4;
  if (E == 1) append_kernel<T_, D, 1><<<n, kThreads, 0, st>>>(g);
  else if (E == 2) append_kernel<T_, D, 2><<<n, kThreads, 0, st>>>(g);
  else append_kernel<T_, D, kSlots><<<n, kThreads, 0, st>>>(g);
  return check_launch();
}

}  // namespace csa

using namespace csa;

extern "C" int hca_paged_append(const void* a, const void* z, int dtype, int B, int T, int D, int m,
                                const int32_t* pos0, const int32_t* lens, const float* carry_in, float* carry_out,
                                void* pool, int N, int P, const int32_t* table, const int32_t* held, int max_pages,
                                const float* weight, float eps, const double* inv_freq, int R, int flags,
                                int32_t* status, csa_stream_t stream) {
  CSA_REQUIRE((T == 0 || (a && z)) && pos0 && carry_in && carry_out && pool && table && held, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(B >= 0 && T >= 0 && m >= 1 && N >= 0 && P >= 1 && max_pages >= 1, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(R >= 0 && R <= D && (R == 0 || inv_freq) && eps >= 0.f, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE((flags & ~(CSA_NORM | CSA_ROPE_INVERSE | CSA_ROPE_HALF)) == 0, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(dtype == CSA_F32 || dtype == CSA_BF16, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE((D == 64 || D == 128 || D == 256) && R % 16 == 0, CSA_ERR_UNSUPPORTED);
  CSA_REQUIRE(m <= 65536 && T <= (1 << 30), CSA_ERR_UNSUPPORTED);     // 31-bit token counts
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
  // blocks a CTA sums at once: as many as its slots hold the runs of
  int E = kSlots;
  while (E > 1 && kSlots / E < g.runs) E /= 2;
  g.ctas_seq = 1 + (T / m + E - 1) / E;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == CSA_F32)
    return D == 64 ? launch_append<float, 64>(g, B, E, st)
                   : D == 128 ? launch_append<float, 128>(g, B, E, st) : launch_append<float, 256>(g, B, E, st);
  return D == 64 ? launch_append<__nv_bfloat16, 64>(g, B, E, st)
                 : D == 128 ? launch_append<__nv_bfloat16, 128>(g, B, E, st) : launch_append<__nv_bfloat16, 256>(g, B, E, st);
}
