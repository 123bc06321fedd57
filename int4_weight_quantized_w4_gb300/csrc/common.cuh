// Device-side helpers shared by the kernels of the int4-weight linear layer.
// sm_103a only: every helper is plain CUDA or inline PTX for that target.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "w4.h"

#define W4_DEV __device__ __forceinline__

namespace w4 {

// ---------------------------------------------------------------------------
// device status word (bounded waits record W4_ERR_TIMEOUT here)
// ---------------------------------------------------------------------------

// Sets *status to `code` once (the first error wins).
W4_DEV void report(unsigned int* status, unsigned int code) {
  if (status != nullptr) atomicCAS(status, 0u, code);
}

// ---------------------------------------------------------------------------
// bit helpers
// ---------------------------------------------------------------------------

W4_DEV uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// (a & b) | c as one LOP3.
W4_DEV uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// (a & b) ^ c as one LOP3.
W4_DEV uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// m ? a : b, bit by bit, as one LOP3.
W4_DEV uint32_t select_bits(uint32_t m, uint32_t a, uint32_t b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(d) : "r"(a), "r"(b), "r"(m));
  return d;
}

// d0 += a * b0 and d1 += a * b1, two fp32 FMAs (round to nearest) in one
// packed instruction.
W4_DEV void fma2(float& d0, float& d1, float a, float b0, float b1) {
  asm("{.reg .b64 d, x, y; mov.b64 d, {%0, %1}; mov.b64 x, {%2, %2}; mov.b64 y, {%3, %4}; "
      "fma.rn.f32x2 d, x, y, d; mov.b64 {%0, %1}, d;}"
      : "+f"(d0), "+f"(d1) : "f"(a), "f"(b0), "f"(b1));
}

// d0 += a0 * b0 and d1 += a1 * b1, packed as fma2.
W4_DEV void fma2v(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{.reg .b64 d, x, y; mov.b64 d, {%0, %1}; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; "
      "fma.rn.f32x2 d, x, y, d; mov.b64 {%0, %1}, d;}"
      : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

W4_DEV float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
W4_DEV float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// fp32 -> bf16 bits, round to nearest even (finite inputs).
W4_DEV uint32_t f32_to_bf16_bits(float f) {
  uint16_t h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(f));
  return h;
}

W4_DEV uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

W4_DEV float half_bits_to_f32(uint32_t h16) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(static_cast<uint16_t>(h16)));
  return f;
}

// ---------------------------------------------------------------------------
// 8-bit activation codes -> exact fp16, k permuted per 8-chunk
// (the operand layout of the W4A8 tensor-core kernel)
// ---------------------------------------------------------------------------

// int8 bytes b0..b7 -> fp16 (b0,b4,b1,b5,b2,b6,b3,b7). (b ^ 0x80) in the low
// mantissa byte of 1024 is 1152 + b; subtracting 1152 leaves b exactly.
W4_DEV uint32_t i8pair(uint32_t u0, uint32_t u1, uint32_t sel) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(and_xor(prmt(u0, u1, sel), 0x00FF00FFu, 0x64806480u)),
      "r"(0x64806480u));
  return d;
}

W4_DEV uint4 widen_i8(uint32_t u0, uint32_t u1) {
  return make_uint4(i8pair(u0, u1, 0x0400u), i8pair(u0, u1, 0x0501u), i8pair(u0, u1, 0x0602u),
                    i8pair(u0, u1, 0x0703u));
}

W4_DEV uint32_t e4m3x2_to_f16x2(uint32_t two_codes) {
  uint32_t d;
  asm("{.reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(d) : "r"(two_codes));
  return d;
}

// e4m3 codes b0..b7 -> fp16 (b0,b4,b1,b5,b2,b6,b3,b7), exactly.
W4_DEV uint4 widen_e4m3(uint32_t u0, uint32_t u1) {
  const uint32_t a = prmt(u0, u1, 0x5140u), b = prmt(u0, u1, 0x7362u);
  return make_uint4(e4m3x2_to_f16x2(a & 0xFFFFu), e4m3x2_to_f16x2(a >> 16), e4m3x2_to_f16x2(b & 0xFFFFu),
                    e4m3x2_to_f16x2(b >> 16));
}

// ---------------------------------------------------------------------------
// per-token quantization: the codes of the IEEE quotient fl(x / s)
// ---------------------------------------------------------------------------

W4_DEV uint32_t e4m3x2_rn(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}

// Packed fp32 pairs: one f32x2 instruction for two results, round to nearest.
W4_DEV void mul2(float& d0, float& d1, float a0, float a1, float b) {
  asm("{.reg .b64 d, x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %4}; mul.rn.f32x2 d, x, y; mov.b64 {%0, %1}, d;}"
      : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b));
}
W4_DEV void mul2v(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{.reg .b64 d, x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 d, x, y; mov.b64 {%0, %1}, d;}"
      : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
W4_DEV void add2(float& d0, float& d1, float a0, float a1, float b) {
  asm("{.reg .b64 d, x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %4}; add.rn.f32x2 d, x, y; mov.b64 {%0, %1}, d;}"
      : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b));
}

// Halfwise larger magnitude of two words of two 16-bit floats (bf16, or fp16
// with kF16); the sign bits of the result carry no meaning.
template <bool kF16>
W4_DEV uint32_t absmax2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (kF16)
    asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The codes of the IEEE quotient fl(x / s). With r = fl(1 / s) and the two
// per-row factors rlo = fl(r (1 - 2^-20)), rhi = fl(r (1 + 2^-20)), the products
// fl(x rlo) and fl(x rhi) are (x / s)(1 -+ 2^-20)(1 + e) with |e| < 3.1 * 2^-24,
// while fl(x / s) = (x / s)(1 + e'), |e'| <= 2^-24: fl(x / s) lies between the
// two products (a tiny x whose products underflow lies with them below every
// rounding boundary). Rounding onto the int8 or e4m3 grid is monotone, so
// where both products give the same code, that is the code of fl(x / s). An
// 8-element chunk in which some element's ends differ takes the IEEE divide
// for all 8: a value within about 2^-20 of a rounding boundary, or a
// near-exact tie, which bf16 inputs make common (0.2 to 0.3% of elements:
// x / amax is a ratio of two 8-bit mantissas). Measured on GB300 against a
// test per pair of elements, and against a per-chunk test with per-pair
// divides inside: one test per chunk is fastest on activations with outlier
// channels and within 5% on tie-heavy rows without them.
//
// A subnormal s (amax below 2^-126 times the code maximum) breaks the relative
// bounds and may overflow 1 / s: there rlo = 0 and rhi = inf, whose ends differ
// on every element, so such rows are quantized with the divide throughout.
struct QuotientBracket {
  float s, rlo, rhi;
};

W4_DEV QuotientBracket quotient_bracket(float s) {
  if (s < 1.17549435e-38f) return {s, 0.f, __int_as_float(0x7f800000)};
  const float r = __frcp_rn(s);
  return {s, r * 0.99999904632568359375f, r * 1.00000095367431640625f};
}

// Activation halves of a word as fp32 (exact): bf16, or fp16 (kF16).
template <bool kF16>
W4_DEV float act_lo(uint32_t w) {
  return kF16 ? half_bits_to_f32(w & 0xFFFFu) : bf16_lo(w);
}
template <bool kF16>
W4_DEV float act_hi(uint32_t w) {
  return kF16 ? half_bits_to_f32(w >> 16) : bf16_hi(w);
}

// The int8 codes clamp(rne(fl(x / s)), -127, 127) of the 8 activations of a
// 16-byte chunk, element i in byte i. Adding 1.5 * 2^23 rounds a value below
// 2^22 in magnitude to an integer (round to nearest even) and leaves that
// integer in the low bits of the sum, its low byte the two's-complement code.
// On the bracket path |x / s| <= 127 (1 + 2^-22) (s normal, |x| <= amax), so
// no code leaves [-127, 127] and no clamp is needed there.
template <bool kF16>
W4_DEV uint2 quant_int8_chunk(const uint4& v, const QuotientBracket& b) {
  constexpr float kMagic = 12582912.f;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[8];
  uint32_t diff = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float xl = act_lo<kF16>(w[i]), xh = act_hi<kF16>(w[i]);
    float l0, l1, h0, h1;
    mul2(l0, l1, xl, xh, b.rlo);
    mul2(h0, h1, xl, xh, b.rhi);
    add2(l0, l1, l0, l1, kMagic);
    add2(h0, h1, h0, h1, kMagic);
    c[2 * i] = __float_as_uint(l0);
    c[2 * i + 1] = __float_as_uint(l1);
    diff |= (c[2 * i] ^ __float_as_uint(h0)) | (c[2 * i + 1] ^ __float_as_uint(h1));
  }
  if (diff != 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float ql = fmaxf(-127.f, fminf(127.f, __fdiv_rn(act_lo<kF16>(w[i]), b.s)));
      const float qh = fmaxf(-127.f, fminf(127.f, __fdiv_rn(act_hi<kF16>(w[i]), b.s)));
      c[2 * i] = __float_as_uint(ql + kMagic);
      c[2 * i + 1] = __float_as_uint(qh + kMagic);
    }
  }
  return make_uint2(prmt(prmt(c[0], c[1], 0x0040u), prmt(c[2], c[3], 0x0040u), 0x5410u),
                    prmt(prmt(c[4], c[5], 0x0040u), prmt(c[6], c[7], 0x0040u), 0x5410u));
}

// The e4m3 codes (satfinite, round to nearest even) of fl(x / s) for the 8
// activations of a 16-byte chunk, element i in byte i.
template <bool kF16>
W4_DEV uint2 quant_e4m3_chunk(const uint4& v, const QuotientBracket& b) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t p[4];
  uint32_t diff = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float xl = act_lo<kF16>(w[i]), xh = act_hi<kF16>(w[i]);
    float l0, l1, h0, h1;
    mul2(l0, l1, xl, xh, b.rlo);
    mul2(h0, h1, xl, xh, b.rhi);
    p[i] = e4m3x2_rn(l0, l1);
    diff |= p[i] ^ e4m3x2_rn(h0, h1);
  }
  if (diff != 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = e4m3x2_rn(__fdiv_rn(act_lo<kF16>(w[i]), b.s), __fdiv_rn(act_hi<kF16>(w[i]), b.s));
  }
  return make_uint2(prmt(p[0], p[1], 0x5410u), prmt(p[2], p[3], 0x5410u));
}

// (d0, d1) = (a0, a1) * (b0, b1) + (c0, c1), packed as fma2.
W4_DEV void fma2x(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{.reg .b64 d, x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7}; "
      "fma.rn.f32x2 d, x, y, z; mov.b64 {%0, %1}, d;}"
      : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
// Per-block quantization: a half-warp holds a block of 128 columns of a row, one
// chunk of 8 per lane. Scale fl(amax / 448), 1 for a block of zeros (which the divide
// would take a slow way through: 1 x 14336 x 4096 12.5 us against 12.4). The quotient of
// a 16-bit amax is never 0; fp32 values below 3e-43 have block_scale_f32.
W4_DEV float block_scale(float amax) { return amax == 0.f ? 1.f : __fdiv_rn(amax, 448.f); }
// 1 also where the quotient is 0: the zeros of such a block would get the code of 0 / 0.
W4_DEV float block_scale_f32(float amax) {
  const float s = block_scale(amax);
  return s == 0.f ? 1.f : s;
}

// (d0, d1) = (a0, a1) * b + (c0, c1), packed as fma2; kDown: rounded down.
template <bool kDown = false>
W4_DEV void fma2c(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
  if constexpr (kDown)
    asm("{.reg .b64 d, x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %4}; mov.b64 z, {%5, %6}; "
        "fma.rm.f32x2 d, x, y, z; mov.b64 {%0, %1}, d;}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
  else
    asm("{.reg .b64 d, x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %4}; mov.b64 z, {%5, %6}; "
        "fma.rn.f32x2 d, x, y, z; mov.b64 {%0, %1}, d;}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}

// The e4m3 codes of the fp32 quotients fl(x0 / s), fl(x1 / s) in the low two
// bytes, with r = fl(1 / s). Division by multiply-add refinement (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// IBM J. Res. Dev. 34(1), 1990): with r the correctly rounded reciprocal and q
// within one ulp of x / s, the remainder x - q s is exact in one FMA and
// fl(q + remainder * r) is the correctly rounded quotient. fl(x r) is within 1.5
// ulp; one step brings it within one, the second rounds it correctly. Holds while
// the remainder does not underflow where it matters: a quotient below 2^-11 has
// code 0 either way, and above that x is at least 2^-11 s and the remainder's last
// bit 2^-48 x, so s >= kRefineMin = 2^-80 is ample. A zero keeps its sign: the remainder
// of -0 has to be -0, since -0 + (+0) r is +0. x - q s of two zeros rounds to -0 downwards,
// and so does every other remainder of 0, which then adds nothing; one that is
// not 0 is exact whatever the direction (the first step's but for a last bit). Of negated x, s and r (kNegated) the signs come
// out with a remainder of +0, rounded to nearest (with every x negated to use that form
// throughout, 32768 x 2048 bf16 took 34.8 us against 33.3). No branch: with the bracket of
// quant_e4m3_chunk half of all warps met a tie of a bf16 ratio somewhere and paid
// 8 divides (146 instructions a chunk, against 80).
// With kSteps = 1 the quotient is within one ulp: for values that are rounded themselves.
constexpr float kRefineMin = 8.27180613e-25f;
template <int kSteps, bool kNegated>
W4_DEV uint32_t quotient2_e4m3(float x0, float x1, float s, float r) {
  float q0, q1, e0, e1;
  mul2(q0, q1, x0, x1, r);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    fma2c<!kNegated>(e0, e1, q0, q1, -s, x0, x1);
    fma2c(q0, q1, e0, e1, r, q0, q1);
  }
  return e4m3x2_rn(q0, q1);
}

// Whether s takes the refinement: not below kRefineMin (a block of values below 4e-22), and finite.
W4_DEV bool scale_refines(float s) { return s >= kRefineMin && s < 1e37f; }

// The codes of 8 values x, or with kNegated of -x, where scale_refines(s).
template <int kSteps = 2, bool kNegated = false>
W4_DEV uint2 quant_e4m3_refined(const float (&x)[8], float s, float r) {
  uint32_t p[4];
  if (kNegated) s = -s, r = -r;
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = quotient2_e4m3<kSteps, kNegated>(x[2 * i], x[2 * i + 1], s, r);
  return make_uint2(prmt(p[0], p[1], 0x5410u), prmt(p[2], p[3], 0x5410u));
}

// The same for any s: out of that range by the IEEE divide.
template <int kSteps = 2, bool kNegated = false>
W4_DEV uint2 quant_e4m3_block(const float (&x)[8], float s, float r) {
  if (scale_refines(s)) return quant_e4m3_refined<kSteps, kNegated>(x, s, r);
  if (kNegated) s = -s;
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = e4m3x2_rn(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s));
  return make_uint2(prmt(p[0], p[1], 0x5410u), prmt(p[2], p[3], 0x5410u));
}

// A chunk's magnitude maximum, and its elements as fp32.
template <bool kF16>
W4_DEV float chunk_max(const uint4& v) {
  const uint32_t m2 = absmax2<kF16>(absmax2<kF16>(v.x, v.y), absmax2<kF16>(v.z, v.w));
  return fmaxf(fabsf(act_lo<kF16>(m2)), fabsf(act_hi<kF16>(m2)));
}
template <bool kF16>
W4_DEV void chunk_f32(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = act_lo<kF16>(w[i]);
    x[2 * i + 1] = act_hi<kF16>(w[i]);
  }
}

// The larger of two numbers; kNaN: NaN where either is (fmaxf drops it).
template <bool kNaN>
W4_DEV float max_of(float a, float b) {
  if constexpr (!kNaN) return fmaxf(a, b);
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The maxima of four blocks over the half-warp, reduced together: lanes trade one
// half of their values for the other at each of the first two steps, which leaves the
// maximum of block u in the lanes with lane % 4 == u.
template <bool kNaN>
W4_DEV float unit_max(const float (&m)[4]) {
  const int lane = threadIdx.x & 31;
  const bool b0 = lane & 1, b1 = lane & 2;
  const float x = max_of<kNaN>(b0 ? m[1] : m[0], __shfl_xor_sync(0xffffffffu, b0 ? m[0] : m[1], 1));
  const float y = max_of<kNaN>(b0 ? m[3] : m[2], __shfl_xor_sync(0xffffffffu, b0 ? m[2] : m[3], 1));
  float z = max_of<kNaN>(b1 ? y : x, __shfl_xor_sync(0xffffffffu, b1 ? x : y, 2));
  z = max_of<kNaN>(z, __shfl_xor_sync(0xffffffffu, z, 4));
  return max_of<kNaN>(z, __shfl_xor_sync(0xffffffffu, z, 8));
}

// This lane's codes and the scale of one block. Every lane of the warp takes part.
template <bool kF16>
W4_DEV void quant_block_half_warp(const uint4& v, uint2& code, float& s) {
  float m = chunk_max<kF16>(v);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  s = block_scale(m);
  float x[8];
  chunk_f32<kF16>(v, x);
  code = quant_e4m3_block(x, s, __frcp_rn(s));
}

// Four blocks of the half-warp at once, chunk v[u] of block u: this lane's codes
// and (in lane l) the scale of block l % 4. Every lane of the warp takes part.
template <bool kF16>
W4_DEV float quant_blocks4(const uint4 (&v)[4], uint2 (&code)[4]) {
  float m[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) m[u] = chunk_max<kF16>(v[u]);
  const float s_mine = block_scale(unit_max<false>(m)), r_mine = __frcp_rn(s_mine);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float s = __shfl_sync(0xffffffffu, s_mine, u, 16), r = __shfl_sync(0xffffffffu, r_mine, u, 16);
    float x[8];
    chunk_f32<kF16>(v[u], x);
    code[u] = quant_e4m3_block(x, s, r);
  }
  return s_mine;
}

// ---------------------------------------------------------------------------
// global memory access
// ---------------------------------------------------------------------------

// 16-byte streaming load that bypasses L1 (each weight byte is read once).
W4_DEV uint4 ld_stream_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

W4_DEV uint4 ld_nc_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// 16-byte load cached in L2 only: sees data another grid wrote, even one
// that finished while this grid was already running.
W4_DEV uint4 ld_cg_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// 16-byte streaming load that keeps nothing in L1, of data that another grid may have
// written while this one was already running (the .nc loads above want data that
// nothing writes for as long as the kernel runs).
W4_DEV uint4 ld_once_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

W4_DEV uint2 ld_nc_v2(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// ---------------------------------------------------------------------------
// mbarrier with bounded waits
// ---------------------------------------------------------------------------

W4_DEV uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

W4_DEV void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(smem_addr(bar)), "r"(count));
}

W4_DEV void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

W4_DEV void mbar_arrive(uint64_t* bar) {
  asm volatile("{.reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0];}" :: "r"(smem_addr(bar)) : "memory");
}

W4_DEV void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("{.reg .b64 st; mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;}"
               :: "r"(smem_addr(bar)), "r"(bytes) : "memory");
}

W4_DEV bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{.reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p;}"
      : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
  return ok != 0;
}

// Waits for phase `parity` of `bar` to complete, polling at most `limit`
// times. Returns false (after recording W4_ERR_TIMEOUT) if it never does.
W4_DEV bool mbar_wait_bounded(uint64_t* bar, uint32_t parity, long long limit, unsigned int* status) {
  for (long long i = 0; i < limit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
  }
  report(status, W4_ERR_TIMEOUT);
  return false;
}

}  // namespace w4
