// qk_norm_rope: per-head RMS norm of queries and the shared raw key, with the
// position rotation, in one pass over the data.
//
//   y = x rsqrt(mean(x^2) + eps) w;   (y0, y1) -> (y0 c - y1 s, y0 s + y1 c)
//
// Bound by HBM: each value is read and written once.  A row is D / 8 lanes of
// 16-byte (bf16) loads, so a warp moves whole rows; the norm is a shuffle
// reduction over those lanes.  The angles depend on the token alone: a CTA
// works on the rows of one token and forms its R / 2 cosines and sines once, in
// shared memory.
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
  int rows, rows_cta, chunks;   // rows per token (H, and one for the key); rows per CTA; CTAs per token
};

constexpr int kNrThreads = 256;

template <typename T_, int D>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int G = D / 8, NG = kNrThreads / G;
  __shared__ float2 cs[D / 2];
  const long long tok = blockIdx.x / a.chunks;
  const int chunk = blockIdx.x - static_cast<int>(tok * a.chunks);
  const int b = static_cast<int>(tok / a.T), t = static_cast<int>(tok - static_cast<long long>(b) * a.T);
  const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
  if (t >= len) return;
  const long long j = static_cast<long long>(a.pos0[b]) + t;
  const bool half = a.flags & CSA_ROPE_HALF;
  for (int i = threadIdx.x; i < a.R / 2; i += kNrThreads)
    cs[i] = cos_sin_at(j * a.pos_step, a.inv_freq[i], a.flags & CSA_ROPE_INVERSE);
  __syncthreads();
  const int l = threadIdx.x % G, g = threadIdx.x / G;
  LaneRope lr;
  load_lane_rope<D>(lr, cs, a.R, half, l);
  const int r0 = chunk * a.rows_cta, r1 = min(r0 + a.rows_cta, a.rows);
  for (int base = r0; base < r1; base += NG) {
    const int r = base + g;
    const bool isq = r < a.H;
    bool ok = r < r1;
    const T_* src = nullptr;
    T_* dst = nullptr;
    if (ok) {
      if (isq) {
        src = static_cast<const T_*>(a.q) + b * a.q_bs + t * a.q_ts + static_cast<long long>(r) * D + l * 8;
        dst = static_cast<T_*>(a.q_out) + ((static_cast<long long>(b) * a.T + t) * a.H + r) * D + l * 8;
      } else {
        src = static_cast<const T_*>(a.kv) + b * a.kv_bs + t * a.kv_ts + l * 8;
        // of the call's tokens only the last kv_cap reach the ring
        long long slot = t;
        if (!a.kv_inplace) {
          if (t < len - a.kv_cap) ok = false;
          slot = j % a.kv_cap;
          if (slot < 0) slot += a.kv_cap;
        }
        dst = static_cast<T_*>(a.kv_out) + (static_cast<long long>(b) * a.kv_cap + slot) * D + l * 8;
      }
    }
    float v[8];
    if (ok) {
      Vec8<T_>::load(src, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    if (a.flags & CSA_NORM) {
      const float sc = row_rms_scale<D>(v, a.eps);
      const float* w = isq ? a.q_w : a.kv_w;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * sc * (w ? w[l * 8 + i] : 1.f);
    }
    rotate8(v, lr, a.R, half);
    if (ok) Vec8<T_>::store(dst, v);
  }
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
  const long long tokens = static_cast<long long>(B) * T;
  const int ng = kNrThreads / (D / 8);
  a.rows_cta = a.rows;
  a.chunks = (a.rows + a.rows_cta - 1) / a.rows_cta;
  (void)ng;
  const long long grid = tokens * a.chunks;
  CSA_REQUIRE(grid < (1ll << 31), CSA_ERR_UNSUPPORTED);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
#define NR(TT, DD) norm_rope_kernel<TT, DD><<<static_cast<unsigned>(grid), kNrThreads, 0, st>>>(a)
  if (dtype == CSA_F32) {
    if (D == 64) NR(float, 64); else if (D == 128) NR(float, 128); else NR(float, 256);
  } else {
    if (D == 64) NR(__nv_bfloat16, 64); else if (D == 128) NR(__nv_bfloat16, 128); else NR(__nv_bfloat16, 256);
  }
#undef NR
  return check_launch();
}
