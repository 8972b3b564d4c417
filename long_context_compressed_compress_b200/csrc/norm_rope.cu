// qk_norm_rope: per-head RMS norm of queries and the shared raw key, with the
// position rotation, in one pass over the data.
//
//   y = x rsqrt(mean(x^2) + eps) w;   (y0, y1) -> (y0 c - y1 s, y0 s + y1 c)
//
// Bound by HBM: each value is read and written once.  A row is D / 8 lanes of
// 16-byte (bf16) loads, so a warp moves whole rows; the norm is a shuffle
// reduction over those lanes.  A warp takes a run of one token's rows: its lanes form
// the cosines and sines they meet once, keep them in registers, and go through
// the rows three or four at a time with all loads under way.  (A CTA-wide table of
// angles in shared memory cost a barrier and half the occupancy: 355 to 646 us for
// 32768 tokens of 64 heads.)
#include <type_traits>

#include "rope.cuh"

namespace csa {

struct NormRopeArgs {
  const void* q;
  const void* kv;
  void* q_out;
  void* kv_out;
  long long q_bs, q_ts, kv_bs, kv_ts;
  const int32_t* pos0;
  const int32_t* lens;
  const double* inv_freq;
  const float* q_w;
  const float* kv_w;
  float eps;
  int T, H, R, pos_step, flags, kv_cap, kv_inplace;
  int rows;              // per token: H, and one for the key
  int chunk;             // rows a warp takes
  uint32_t chunks;       // warps per token
  uint32_t items;
};

// (32768 tokens of 64 heads: 195 us with 256 threads a CTA.)
constexpr int kNrThreads = 128;

template <typename T_, int D, bool HALF>
__global__ void __launch_bounds__(kNrThreads, sizeof(T_) == 2 ? 8 : 6) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int G = D / 8, RW = 32 / G;       // lanes a row, rows a warp
  // loads under way (64233 tokens of 16 heads, split halves: 123 us with four, 112 with three;
  // neighbours 109 and 106, but 64 heads 191 and 195)
  constexpr int kFlight = HALF ? 3 : 4;
  const int lane = threadIdx.x & 31, l = lane % G, sub = lane / G;
  const uint32_t item = blockIdx.x * (kNrThreads / 32) + (threadIdx.x >> 5);
  if (item >= a.items) return;
  const uint32_t tok32 = item / a.chunks;
  const long long tok = tok32;
  const int r0 = static_cast<int>(item - tok32 * a.chunks) * a.chunk, r1 = min(r0 + a.chunk, a.rows);
  const int b = static_cast<int>(tok32 / a.T), t = static_cast<int>(tok32 - static_cast<uint32_t>(b) * a.T);
  const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
  if (t >= len) return;
  const long long j = static_cast<long long>(a.pos0[b]) + t;
  const LaneRuns at = lane_runs<D>(l, a.R, HALF);
  const int apart = at.b - at.a;
  const T_* qs = static_cast<const T_*>(a.q) + b * a.q_bs + t * a.q_ts + at.a;
  T_* qd = static_cast<T_*>(a.q_out) + tok * a.H * D + at.a;
  const T_* ks = static_cast<const T_*>(a.kv) + b * a.kv_bs + t * a.kv_ts + at.a;
  T_* kd = nullptr;                           // of the call's tokens only the last kv_cap reach the ring
  if (a.kv_inplace) {
    kd = static_cast<T_*>(a.kv_out) + tok * D + at.a;
  } else if (a.kv_out && t >= len - a.kv_cap) {
    long long slot = j >= 0 && j < (1ll << 31) ? static_cast<uint32_t>(j) % static_cast<uint32_t>(a.kv_cap) : j % a.kv_cap;
    if (slot < 0) slot += a.kv_cap;
    kd = static_cast<T_*>(a.kv_out) + (static_cast<long long>(b) * a.kv_cap + slot) * D + at.a;
  }

  Raw8<T_, HALF> raw[kFlight];
  auto fetch = [&](int base) {
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int r = base + i * RW + sub;
      if (r < r1) raw[i].load(r < a.H ? qs + static_cast<long long>(r) * D : ks, apart);
      else raw[i].zero();
    }
  };
  fetch(r0);
  LaneRope lr;
  if (a.R > 0) lane_rope<D>(lr, j * a.pos_step, a.inv_freq, a.R, a.flags & CSA_ROPE_INVERSE, l);
  else lr.active = false;
  const bool norm = a.flags & CSA_NORM;
  float w[8];
  weights8(norm ? a.q_w : nullptr, at, w);
  for (int base = r0; base < r1; base += kFlight * RW) {
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      if (base + i * RW >= r1) break;
      const int r = base + i * RW + sub;
      float v[8];
      raw[i].get(v);
      if (norm) {
        const float sc = row_rms_scale<D>(v, a.eps);
        if (r < a.H) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= sc * w[e];
        } else {
          float kw[8];
          weights8(a.kv_w, at, kw);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= sc * kw[e];
        }
      }
      rotate8<HALF>(v, lr);
      if (r < r1) {
        T_* d = r < a.H ? qd + static_cast<long long>(r) * D : kd;
        if (d) store8<HALF>(d, apart, v);
      }
    }
    if (base + kFlight * RW < r1) fetch(base + kFlight * RW);
  }
}

// Tokens of no more rows than a warp holds (the key alone, one head and the key): a warp
// takes TOK tokens, RW / TOK rows of each, and a token's lanes form its angles, which
// bound such calls.  (293184 tokens of a head and a key, D = 64, split halves: 58 us, 203
// with a token a warp.)
template <typename T_, int D, bool HALF, int TOK>
__global__ void __launch_bounds__(kNrThreads, 8) norm_rope_few_kernel(const NormRopeArgs a) {
  constexpr int G = D / 8, RW = 32 / G, RP = RW / TOK;
  const int lane = threadIdx.x & 31, l = lane % G, r = lane / G % RP;
  const uint32_t item = blockIdx.x * (kNrThreads / 32) + (threadIdx.x >> 5);
  if (item * TOK >= a.items) return;
  const uint32_t tok = min(item * TOK + lane / (G * RP), a.items - 1);
  const bool own = item * TOK + lane / (G * RP) < a.items;
  const uint32_t b = tok / static_cast<uint32_t>(a.T);
  const int t = static_cast<int>(tok - b * a.T), len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
  const LaneRuns at = lane_runs<D>(l, a.R, HALF);
  const int apart = at.b - at.a;
  const bool live = own && t < len && r < a.rows, is_q = r < a.H;
  const long long j = static_cast<long long>(a.pos0[b]) + t;
  const T_* s = (is_q ? static_cast<const T_*>(a.q) + b * a.q_bs + t * a.q_ts + r * D
                      : static_cast<const T_*>(a.kv) + b * a.kv_bs + t * a.kv_ts) + at.a;
  T_* d = nullptr;
  if (is_q) {
    d = static_cast<T_*>(a.q_out) + (static_cast<long long>(tok) * a.H + r) * D + at.a;
  } else if (a.kv_inplace) {
    d = static_cast<T_*>(a.kv_out) + static_cast<long long>(tok) * D + at.a;
  } else if (t >= len - a.kv_cap) {
    long long slot = j >= 0 && j < (1ll << 31) ? static_cast<uint32_t>(j) % static_cast<uint32_t>(a.kv_cap) : j % a.kv_cap;
    if (slot < 0) slot += a.kv_cap;
    d = static_cast<T_*>(a.kv_out) + (static_cast<long long>(b) * a.kv_cap + slot) * D + at.a;
  }
  Raw8<T_, HALF> raw;
  if (live) raw.load(s, apart);
  else raw.zero();
  LaneRope lr;
  if (a.R > 0) lane_rope<D, 32 / TOK>(lr, j * a.pos_step, a.inv_freq, a.R, a.flags & CSA_ROPE_INVERSE, l);
  else lr.active = false;
  float v[8];
  raw.get(v);
  if (a.flags & CSA_NORM) {
    const float sc = row_rms_scale<D>(v, a.eps);
    float w8[8];
    weights8(is_q ? a.q_w : a.kv_w, at, w8);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= sc * w8[e];
  }
  rotate8<HALF>(v, lr);
  if (live && d) store8<HALF>(d, apart, v);
}

// [lo, hi) bytes of a strided tensor
struct Span {
  uintptr_t lo, hi;
};
inline Span span_of(const void* p, long long bs, long long ts, long long row, int B, int T, int es) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + static_cast<uintptr_t>(((B - 1) * bs + (T - 1) * ts + row) * es)};
}
inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

template <typename T_, int D>
int launch_norm_rope(NormRopeArgs& a, cudaStream_t st) {
  // A run of rows long enough that the angles (some 100 instructions a lane) are a
  // small part of it, but short where there are few rows, to spread them over the SMs.
  constexpr int RW = 32 / (D / 8);
  const long long tokens = a.items;
  if (a.rows <= RW) {
    const auto few = [&](auto tok) {
      constexpr int TOK = decltype(tok)::value;
      const uint32_t warps = (a.items + TOK - 1) / TOK, grid = (warps + kNrThreads / 32 - 1) / (kNrThreads / 32);
      if (a.flags & CSA_ROPE_HALF) norm_rope_few_kernel<T_, D, true, TOK><<<grid, kNrThreads, 0, st>>>(a);
      else norm_rope_few_kernel<T_, D, false, TOK><<<grid, kNrThreads, 0, st>>>(a);
      return check_launch();
    };
    if (a.rows == 1) return few(std::integral_constant<int, RW>());
    if (RW == 4 && a.rows == 2) return few(std::integral_constant<int, RW == 4 ? 2 : 1>());
    return few(std::integral_constant<int, 1>());
  }
  int iters = 16;
  while (iters > 1 && tokens * ((a.rows + iters * RW - 1) / (iters * RW)) < 148 * 32) iters /= 2;
  a.chunk = iters * RW;
  a.chunks = (a.rows + a.chunk - 1) / a.chunk;
  a.chunk = ((a.rows + a.chunks - 1) / a.chunks + RW - 1) / RW * RW;     // evenly
  CSA_REQUIRE(tokens * a.chunks < (1ll << 31), CSA_ERR_UNSUPPORTED);
  a.items = static_cast<uint32_t>(tokens * a.chunks);
  const uint32_t grid = (a.items + kNrThreads / 32 - 1) / (kNrThreads / 32);
  if (a.flags & CSA_ROPE_HALF) norm_rope_kernel<T_, D, true><<<grid, kNrThreads, 0, st>>>(a);
  else norm_rope_kernel<T_, D, false><<<grid, kNrThreads, 0, st>>>(a);
  return check_launch();
}

}  // namespace csa

using namespace csa;

extern "C" int qk_norm_rope(const void* q, int64_t q_bstride, int64_t q_tstride, const void* kv, int64_t kv_bstride,
                            int64_t kv_tstride, int dtype, int B, int T, int H, int D, const int32_t* q_pos0,
                            const int32_t* lens, int pos_step, const double* inv_freq, int R, const float* q_weight,
                            const float* kv_weight, float eps, int flags, void* q_out, void* kv_out, int kv_cap,
                            csa_stream_t stream) {
  CSA_REQUIRE((q != nullptr) == (q_out != nullptr) && (kv != nullptr) == (kv_out != nullptr), CSA_ERR_INVALID_ARG);
  CSA_REQUIRE((q || kv) && q_pos0, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(B >= 0 && T >= 0 && H >= 0 && R >= 0 && R <= D && (R == 0 || inv_freq), CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(!kv || kv_cap >= 1, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(dtype == CSA_F32 || dtype == CSA_BF16, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE((flags & ~(CSA_NORM | CSA_ROPE_INVERSE | CSA_ROPE_HALF)) == 0 && eps >= 0.f, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE((D == 64 || D == 128 || D == 256) && R % 16 == 0, CSA_ERR_UNSUPPORTED);
  const long long hd = static_cast<long long>(H) * D;
  CSA_REQUIRE(!q || (q_tstride >= 0 && q_bstride >= 0), CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(!kv || (kv_tstride >= 0 && kv_bstride >= 0), CSA_ERR_INVALID_ARG);
  CSA_REQUIRE((!q || (q_bstride % 8 == 0 && q_tstride % 8 == 0)) &&
                  (!kv || (kv_bstride % 8 == 0 && kv_tstride % 8 == 0)),
              CSA_ERR_ALIGNMENT);
  CSA_REQUIRE(aligned16(q) && aligned16(kv) && aligned16(q_out) && aligned16(kv_out) && aligned16(q_weight) &&
                  aligned16(kv_weight),
              CSA_ERR_ALIGNMENT);
  if (B == 0 || T == 0 || (!kv && H == 0)) return CSA_OK;
  const int es = dtype == CSA_F32 ? 4 : 2;
  const bool do_q = q && H > 0;
  bool kv_inplace = false;
  {
    const Span none{0, 0};
    const Span qi = do_q ? span_of(q, q_bstride, q_tstride, hd, B, T, es) : none;
    const Span qo = do_q ? span_of(q_out, T * hd, hd, hd, B, T, es) : none;
    const Span ki = kv ? span_of(kv, kv_bstride, kv_tstride, D, B, T, es) : none;
    const Span ko = kv ? span_of(kv_out, static_cast<long long>(kv_cap) * D, D, D, B, kv_cap, es) : none;
    const bool q_same = q == q_out && (T == 1 || q_tstride == hd) && (B == 1 || q_bstride == T * hd);
    kv_inplace = kv && kv == kv_out && kv_cap == T && (T == 1 || kv_tstride == D) &&
                 (B == 1 || kv_bstride == static_cast<long long>(T) * D);
    CSA_REQUIRE(!do_q || q_same || !overlap(qi, qo), CSA_ERR_INVALID_ARG);
    CSA_REQUIRE(!kv || kv_inplace || !overlap(ki, ko), CSA_ERR_INVALID_ARG);
    CSA_REQUIRE(!overlap(qi, ko) && !overlap(ki, qo) && !overlap(qo, ko), CSA_ERR_INVALID_ARG);
  }
  NormRopeArgs a;
  a.q = q; a.kv = kv; a.q_out = q_out; a.kv_out = kv_out;
  a.q_bs = q_bstride; a.q_ts = q_tstride; a.kv_bs = kv_bstride; a.kv_ts = kv_tstride;
  a.pos0 = q_pos0; a.lens = lens; a.inv_freq = inv_freq; a.q_w = q_weight; a.kv_w = kv_weight; a.eps = eps;
  a.T = T; a.H = do_q ? H : 0; a.R = R; a.pos_step = pos_step; a.flags = flags; a.kv_cap = kv_cap;
  a.kv_inplace = kv_inplace;
  a.rows = a.H + (kv ? 1 : 0);
  CSA_REQUIRE(static_cast<long long>(B) * T < (1ll << 31), CSA_ERR_UNSUPPORTED);
  a.items = static_cast<uint32_t>(B) * T;       // (tokens, so far)
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == CSA_F32)
    return D == 64 ? launch_norm_rope<float, 64>(a, st)
                   : D == 128 ? launch_norm_rope<float, 128>(a, st) : launch_norm_rope<float, 256>(a, st);
  return D == 64 ? launch_norm_rope<__nv_bfloat16, 64>(a, st)
                 : D == 128 ? launch_norm_rope<__nv_bfloat16, 128>(a, st) : launch_norm_rope<__nv_bfloat16, 256>(a, st);
}
