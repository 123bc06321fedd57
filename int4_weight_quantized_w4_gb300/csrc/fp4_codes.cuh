// Codes and scales of microscaled 4-bit floats, 16 elements a thread: what the
// quantizers and the product that quantizes few rows itself share.
#pragma once

#include "common.cuh"

namespace w4 {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u;

// Eight e2m1 codes of eight floats (round to nearest even, held to +-6), element i in nibble i.
W4_DEV uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t d;
  asm("{.reg .b8 a, b, c, d; cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3; "
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7; mov.b32 %0, {a, b, c, d};}"
      : "=r"(d) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return d;
}

// Codes of fl(x / d), with r = fl(1 / d): the quotient by multiply-add refinement as
// quotient2_e4m3, where `refines`: d takes it (scale_refines) and no quotient is beyond 4096,
// as where the block's scale was held at 448 (one that overflows would come out of the
// refinement as NaN, which has lost its sign). A quotient below 2^-3 has code 0 or -0 either
// way, so the lower bounds of the e4m3 form are ample.
W4_DEV uint32_t quotients_e2m1(const float (&x)[8], float d, float r, bool refines) {
  float q[8];
  if (refines) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float q0, q1, e0, e1;
      mul2(q0, q1, x[i], x[i + 1], r);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        fma2c<true>(e0, e1, q0, q1, -d, x[i], x[i + 1]);
        fma2c(q0, q1, e0, e1, r, q0, q1);
      }
      q[i] = q0, q[i + 1] = q1;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(x[i], d);
  }
  return e2m1x8(q);
}

// Halfwise maximum of magnitude bits: NaNs are above infinities, those above numbers.
W4_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// fl(fl(a / 6) / g) up to what e4m3 makes of it, by multiply-add refinement (as
// quotient2_e4m3) where no remainder can underflow or overflow; else by IEEE divides.
W4_DEV float block_quotient(float a, float g) {
  constexpr float kSixth = 0.166666672f;   // fl(1 / 6)
  if (!(a > 1e-25f && a < 1e30f && scale_refines(g))) return __fdiv_rn(__fdiv_rn(a, 6.f), g);
  float v = a * kSixth;
  v = fmaf(fmaf(v, -6.f, a), kSixth, v);
  const float r = __frcp_rn(g);
  float q = v * r;
  if (q < 4096.f) {   // others are held at 448
    q = fmaf(fmaf(q, -g, v), r, q);
    q = fmaf(fmaf(q, -g, v), r, q);
  }
  return q;
}

// Scale byte and codes of 16 elements; bits: those of the block's largest magnitude.
// kNv: the block is this thread's; else it is two lanes'.
template <bool kNv>
W4_DEV uint32_t block_codes(const float (&x)[2][8], uint32_t bits, float g, uint2& code) {
  if constexpr (kNv) {
    if (bits >= kInfBits) {
      code = make_uint2(0, 0);
      return 0x7F;
    }
    const float v = block_quotient(__uint_as_float(bits), g);
    const uint32_t s8 = e4m3x2_rn(v, 0.f) & 0xFFu;
    const float s = half_bits_to_f32(e4m3x2_to_f16x2(s8) & 0xFFFFu);
    const float d = s * g;
    if (d > 0.f) {
      const float r = __frcp_rn(d);
      const bool refines = scale_refines(d) && __uint_as_float(bits) * r < 4096.f;
      code.x = quotients_e2m1(x[0], d, r, refines);
      code.y = quotients_e2m1(x[1], d, r, refines);
    } else {
      code = make_uint2(0, 0);
    }
    return s8;
  } else {
    if (bits >= kInfBits) {
      code = make_uint2(0, 0);
      return 0xFF;
    }
    const uint32_t b = max(static_cast<int>(bits >> 23) - 2, 0);   // floor(log2 amax) - 2 + 127
    const float f = __uint_as_float((254u - b) << 23);
    float y[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) mul2(y[i], y[i + 1], x[h][i], x[h][i + 1], f);
      (h ? code.y : code.x) = e2m1x8(y);
    }
    return b;
  }
}

W4_DEV void load32(const uint4* p, bool wide, uint4 (&v)[2]) {
  if (wide) {
    ld_once_v8(p, v[0], v[1]);
  } else {
    v[0] = ld_once_v4(p);
    v[1] = ld_once_v4(p + 1);
  }
}

// 16 activations as fp32; returns the magnitude bits of the largest.
template <bool kF16>
W4_DEV uint32_t widen16(const uint4 (&v)[2], float (&f)[2][8]) {
  constexpr uint32_t kMag = 0x7FFF7FFFu;
  uint32_t m = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    m = max_u16x2(max_u16x2(m, v[h].x & kMag), v[h].y & kMag);
    m = max_u16x2(max_u16x2(m, v[h].z & kMag), v[h].w & kMag);
    chunk_f32<kF16>(v[h], f[h]);
  }
  m = max(m & 0xFFFFu, m >> 16);
  return __float_as_uint(act_lo<kF16>(m));   // fp16 infinities and NaNs become fp32's
}

}  // namespace
}  // namespace w4
