// Row norm and position rotation shared by qk_norm_rope and the paged append:
// a row of D values lies in D / 8 consecutive lanes of a warp, 8 values a lane.
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

// 8 values as loaded.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float v[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float v[8]) const {
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
    v[4] = __uint_as_float(u.z << 16); v[5] = __uint_as_float(u.z & 0xffff0000u);
    v[6] = __uint_as_float(u.w << 16); v[7] = __uint_as_float(u.w & 0xffff0000u);
  }
};

// The lane's share of the rotation: the cos and sin that its 8 values meet.
// Interleaved pairs use the first four; split halves one per value.
struct LaneRope {
  float c[8], s[8];
  bool active, second;   // the lane's values are rotated; they are the pairs' second halves
};
// Lane l of a row at angle pos * inv_freq, the same in each LG lanes.  Every lane forms
// the angles of pairs x, x + LG, .. (x = lane % LG; one for R = 64 of a whole warp) and
// takes those it meets from the others: the 64-bit arithmetic is most of a short call.
template <int D, bool HALF, int LG = 32>
__device__ __forceinline__ void lane_rope(LaneRope& lr, long long pos, const double* inv_freq, int R, bool inverse,
                                          int l) {
  constexpr int N = HALF ? 8 : 4;
  const int lane = threadIdx.x & 31, x = lane & (LG - 1), pairs = R / 2;
  const int i0 = l * 8 - (D - R);   // the lane's first value within the rotated dims
  lr.active = i0 >= 0 && R > 0;
  lr.second = HALF && i0 >= R / 2;
  const int p0 = !lr.active ? 0 : HALF ? (lr.second ? i0 - R / 2 : i0) : i0 / 2;
#pragma unroll
  for (int k = 0; k < D / 2 / LG; ++k) {
    if (LG * k >= pairs) break;
    float2 mine = make_float2(1.f, 0.f);
    if (LG * k + x < pairs) mine = cos_sin_at(pos, inv_freq[LG * k + x], inverse);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int from = (lane - x) + ((p0 + i) & (LG - 1));
      const float c = __shfl_sync(0xffffffffu, mine.x, from), s = __shfl_sync(0xffffffffu, mine.y, from);
      if (k == 0 || (p0 + i) / LG == k) { lr.c[i] = c; lr.s[i] = s; }
    }
  }
}
// The same where the warp's rows are at different positions: a lane forms what it meets.
template <int D, bool HALF>
__device__ __forceinline__ void lane_rope_alone(LaneRope& lr, long long pos, const double* inv_freq, int R, bool inverse,
                                                int l) {
  const int i0 = l * 8 - (D - R);
  lr.active = i0 >= 0 && R > 0;
  lr.second = HALF && i0 >= R / 2;
  if (!lr.active) return;
  const int p0 = HALF ? (lr.second ? i0 - R / 2 : i0) : i0 / 2;
#pragma unroll
  for (int i = 0; i < (HALF ? 8 : 4); ++i) {
    const float2 t = cos_sin_at(pos, inv_freq[p0 + i], inverse);
    lr.c[i] = t.x;
    lr.s[i] = t.y;
  }
}
// Rotates the lane's 8 values in place (every lane of the warp takes part).
template <bool HALF>
__device__ __forceinline__ void rotate8(float v[8], const LaneRope& lr, int R) {
  if (HALF) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the partner value sits R / 2 dims away: R / 16 lanes
      const int src = (threadIdx.x & 31) + (lr.second ? -(R / 16) : (R / 16));
      const float o = __shfl_sync(0xffffffffu, v[i], lr.active ? src : (threadIdx.x & 31));
      if (lr.active) v[i] = lr.second ? fmaf(v[i], lr.c[i], o * lr.s[i]) : fmaf(v[i], lr.c[i], -o * lr.s[i]);
    }
  } else if (lr.active) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[2 * i], y = v[2 * i + 1];
      v[2 * i] = fmaf(x, lr.c[i], -y * lr.s[i]);
      v[2 * i + 1] = fmaf(x, lr.s[i], y * lr.c[i]);
    }
  }
}

}  // namespace csa
