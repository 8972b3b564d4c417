// Row norm and position rotation shared by qk_norm_rope and the paged append:
// a row of D values lies in D / 8 consecutive lanes of a warp, 8 values a lane.
#pragma once

#include "common.cuh"

namespace csa {

// cos and sin of pos * f (f in radians).  The product and its reduction to the
// nearest quarter turn are in 64 bits: at positions of 2^20 a 32-bit angle
// would be off by 2^-4 rad.  What is left, within an eighth of a turn, rounds to
// fp32 with an error below 2^-28 turns, under fp32's own rounding of the result.
__device__ __forceinline__ float2 cos_sin_at(long long pos, double f, bool inverse) {
  const double turns = static_cast<double>(pos) * f * 0.15915494309189533577;
  const double r = turns - rint(turns);
  const double k = rint(4.0 * r);
  float s, c;
  sincospif(static_cast<float>(2.0 * (r - 0.25 * k)), &s, &c);
  const int q = static_cast<int>(k) & 3;
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

// The lane's share of the rotation: the cos and sin that its 8 values meet.
// Interleaved pairs use the first four; split halves one per value.
struct LaneRope {
  float c[8], s[8];
  bool active, second;   // the lane's values are rotated; they are the pairs' second halves
};
// Reads the row's table cs[R / 2] of (cos, sin).
template <int D>
__device__ __forceinline__ void load_lane_rope(LaneRope& lr, const float2* cs, int R, bool half, int l) {
  const int i0 = l * 8 - (D - R);   // the lane's first value within the rotated dims
  lr.active = i0 >= 0 && R > 0;
  lr.second = half && i0 >= R / 2;
  if (!lr.active) return;
  if (half) {
    const int p0 = lr.second ? i0 - R / 2 : i0;
#pragma unroll
    for (int i = 0; i < 8; ++i) { const float2 t = cs[p0 + i]; lr.c[i] = t.x; lr.s[i] = t.y; }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) { const float2 t = cs[i0 / 2 + i]; lr.c[i] = t.x; lr.s[i] = t.y; }
  }
}
// Rotates the lane's 8 values in place (every lane of the warp takes part).
__device__ __forceinline__ void rotate8(float v[8], const LaneRope& lr, int R, bool half) {
  if (half) {
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
