// E4M3 codes with a scale: the rules that the cache write and the norm's 8-bit output share.
#pragma once

#include "common.cuh"

namespace smla {

// The scale of a block whose largest magnitude is amax: 1 for an all-zero block, else fl32(amax / 448)
// or (SMLA_SCALE_POW2) the smallest power of two that is no less. A quotient that rounds to 0 (below 2^-150, of the norm's fp32
// values only: bf16 ones start at 2^-133) counts as fp32's smallest number, so that no scale is 0.
__device__ __forceinline__ float block_scale(float amax, int scale_mode) {
  if (!(amax > 0.f)) return 1.f;
  const float ratio = fmaxf(__fdiv_rn(amax, 448.f), 0x1p-149f);
  if (scale_mode != SMLA_SCALE_POW2) return ratio;
  int e;
  const float m = frexpf(ratio, &e);  // ratio = m * 2^e, m in [0.5, 1)
  return (m == 0.5f) ? ratio : ldexpf(1.f, e);
}

// x / scale for the E4M3 conversion. Where scale is a power of two in [2^-126, 2^126] its
// reciprocal is exact, so x * (1 / scale) is the same real number x / scale rounded once: the
// same fp32 value as the correctly rounded division, for every x. Otherwise divide.
struct ScaleDiv {
  float scale, inv;
  bool exact;
  __device__ __forceinline__ explicit ScaleDiv(float sc) : scale(sc) {
    const uint32_t b = __float_as_uint(sc);
    exact = (b & 0x007fffffu) == 0u && sc >= 0x1p-126f && sc <= 0x1p126f;
    inv = exact ? __frcp_rn(sc) : 0.f;
  }
  // E4M3 codes of x[0..2n) / scale, two per 16-bit word: one branch for the whole run
  template <int N>
  __device__ __forceinline__ void codes(const float* x, uint16_t* out) const {
    if (exact) {
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = f32x2_to_e4m3x2(__fmul_rn(x[2 * i], inv), __fmul_rn(x[2 * i + 1], inv));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        out[i] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale));
    }
  }
  // The same codes, with three instructions a value in place of a division: with y the correctly rounded reciprocal of the
  // scale, q = x y and r = x - q scale (exact in one fused multiply-add), q + r y rounds to the correctly rounded quotient
  // (Markstein, IBM Journal of Research and Development 34, 1990). Quotients too small for that round to code 0 all the same.
  // The remainder is taken as -r: with it zeros of either sign come out as they are, as from the division.
  template <int N>
  __device__ __forceinline__ void codes_by_reciprocal(const float* x, uint16_t* out) const {
    if (!exact && scale >= 0x1p-60f && scale <= 0x1p60f) {
      const float y = __frcp_rn(scale);
      auto quotient = [&](float v) {
        const float q = __fmul_rn(v, y);
        return __fmaf_rn(-__fmaf_rn(q, scale, -v), y, q);
      };
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = f32x2_to_e4m3x2(quotient(x[2 * i]), quotient(x[2 * i + 1]));
    } else {
      codes<N>(x, out);
    }
  }
};

}  // namespace smla
