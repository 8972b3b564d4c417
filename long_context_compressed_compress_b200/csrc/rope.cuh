// Row norm and position rotation shared by qk_norm_rope and the paged append:
// a row of D values lies in D / 8 consecutive lanes of a warp, 8 values a lane, as two
// runs of four.  The runs are neighbours, but for split halves (pairs (i, i + R / 2)) a
// rotated lane has the same four places of both halves: a pair is in one lane.  (With
// neighbours and the partners fetched by shuffles 64233 tokens of 16 heads took 168
// us for 123.)
#pragma once

#include "common.cuh"

namespace csa {

// cos and sin of pos * f (f in radians).  The product and its reduction to the
// nearest quarter turn are in 64 bits: at positions of 2^20 a 32-bit angle
// would be off by 2^-4 rad.  (Adding and taking away 1.5 * 2^52 rounds to an integer, whose
// low bits are then the sum's; for angles below 2^49 turns.)  What is left, within an
// eighth of a turn, rounds to fp32, and there both functions are their Taylor series: the
// terms left out are below 2^-28 of the result.  (With rint and sincospif 293184
// tokens of a head and a key, D = 128, took 112 us for 107.)
__device__ __forceinline__ float2 cos_sin_at(long long pos, double f, bool inverse) {
  const double quarters = static_cast<double>(pos) * f * (4.0 * 0.15915494309189533577);
  const double m = quarters + 6755399441055744.0;
  const int q = __double2loint(m) & 3;
  const float y = static_cast<float>(quarters - (m - 6755399441055744.0)) * 1.57079632679489662f, z = y * y;
  float s = fmaf(z, 1.f / 362880.f, -1.f / 5040.f), c = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  s = fmaf(z, s, 1.f / 120.f);
  c = fmaf(z, c, -1.f / 720.f);
  s = fmaf(z, s, -1.f / 6.f);
  c = fmaf(z, c, 1.f / 24.f);
  s = fmaf(y * z, s, y);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  float cs = (q & 1) ? s : c, sn = (q & 1) ? c : s;
  if (q == 1 || q == 2) cs = -cs;
  if (q >= 2) sn = -sn;
  return make_float2(cs, inverse ? -sn : sn);
}

// 1 / sqrt(mean(x^2) + eps) of the row, in every lane of it.
template <int D>
__device__ __forceinline__ float row_rms_scale(const float v[8], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return rsqrtf(ss * (1.0f / D) + eps);
}

// Where lane l's runs begin.
struct LaneRuns {
  int a, b;
};
template <int D>
__device__ __forceinline__ LaneRuns lane_runs(int l, int R, bool half) {
  const int i = l - (D - R) / 8;       // the lane's place among the rotated ones
  if (!half || i < 0) return {l * 8, l * 8 + 4};
  return {D - R + 4 * i, D - R / 2 + 4 * i};
}

// 8 values as loaded: the run at p and the one `apart` behind it (4, known, unless SPLIT).
template <typename T, bool SPLIT> struct Raw8;
template <bool SPLIT> struct Raw8<float, SPLIT> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int apart) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + (SPLIT ? apart : 4));
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float v[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <bool SPLIT> struct Raw8<__nv_bfloat16, SPLIT> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int apart) {
    if (SPLIT) {
      const uint2 x = *reinterpret_cast<const uint2*>(p), y = *reinterpret_cast<const uint2*>(p + apart);
      u = make_uint4(x.x, x.y, y.x, y.y);
    } else {
      u = *reinterpret_cast<const uint4*>(p);
    }
  }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float v[8]) const {
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
    v[4] = __uint_as_float(u.z << 16); v[5] = __uint_as_float(u.z & 0xffff0000u);
    v[6] = __uint_as_float(u.w << 16); v[7] = __uint_as_float(u.w & 0xffff0000u);
  }
};
template <bool SPLIT>
__device__ __forceinline__ void store8(float* p, int apart, const float v[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + (SPLIT ? apart : 4)) = make_float4(v[4], v[5], v[6], v[7]);
}
template <bool SPLIT>
__device__ __forceinline__ void store8(__nv_bfloat16* p, int apart, const float v[8]) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  if (SPLIT) {
    *reinterpret_cast<uint2*>(p) = make_uint2(u.x, u.y);
    *reinterpret_cast<uint2*>(p + apart) = make_uint2(u.z, u.w);
  } else {
    *reinterpret_cast<uint4*>(p) = u;
  }
}
// The lane's weights (fp32, or ones).
__device__ __forceinline__ void weights8(const float* w, const LaneRuns& at, float v[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 1.f;
  if (w == nullptr) return;
  Raw8<float, true> r;
  r.load(w + at.a, at.b - at.a);
  r.get(v);
}

// The lane's share of the rotation: the cos and sin of its four pairs.
struct LaneRope {
  float c[4], s[4];
  bool active;           // the lane's values are rotated
};
// Lane l of a row at angle pos * inv_freq, the same in each LG lanes.  Every lane forms
// the angles of pairs x, x + LG, .. (x = lane % LG; one for R = 64 of a whole warp) and
// takes those it meets from the others: the 64-bit arithmetic is most of a short call.
template <int D, int LG = 32>
__device__ __forceinline__ void lane_rope(LaneRope& lr, long long pos, const double* inv_freq, int R, bool inverse,
                                          int l) {
  const int lane = threadIdx.x & 31, x = lane & (LG - 1), pairs = R / 2;
  const int i = l - (D - R) / 8, p0 = max(i, 0) * 4;      // its first pair
  lr.active = i >= 0 && R > 0;
#pragma unroll
  for (int k = 0; k < D / 2 / LG; ++k) {
    if (LG * k >= pairs) break;
    float2 mine = make_float2(1.f, 0.f);
    if (LG * k + x < pairs) mine = cos_sin_at(pos, inv_freq[LG * k + x], inverse);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int from = (lane - x) + ((p0 + e) & (LG - 1));
      const float c = __shfl_sync(0xffffffffu, mine.x, from), s = __shfl_sync(0xffffffffu, mine.y, from);
      if (k == 0 || (p0 + e) / LG == k) { lr.c[e] = c; lr.s[e] = s; }
    }
  }
}
// The same where the warp's rows are at different positions: a lane forms what it meets
// (fewer registers than sharing them within a row).
template <int D>
__device__ __forceinline__ void lane_rope_alone(LaneRope& lr, long long pos, const double* inv_freq, int R, bool inverse,
                                                int l) {
  const int i = l - (D - R) / 8;
  lr.active = i >= 0 && R > 0;
  if (!lr.active) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 t = cos_sin_at(pos, inv_freq[4 * i + e], inverse);
    lr.c[e] = t.x;
    lr.s[e] = t.y;
  }
}
// Rotates the lane's 8 values in place.
template <bool HALF>
__device__ __forceinline__ void rotate8(float v[8], const LaneRope& lr) {
  if (!lr.active) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float& x = v[HALF ? e : 2 * e];
    float& y = v[HALF ? e + 4 : 2 * e + 1];
    const float x0 = x, y0 = y;
    x = fmaf(x0, lr.c[e], -y0 * lr.s[e]);
    y = fmaf(x0, lr.s[e], y0 * lr.c[e]);
  }
}

}  // namespace csa
