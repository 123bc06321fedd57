// Activation quantization for the fp8 block-scaled layer: e4m3 codes with one
// fp32 scale per row and 128 columns.
//
// Per row and block b of 128 columns (the last one may be shorter):
//   amax = max |x|;  s = amax / 448 (IEEE fp32 divide; s = 1 where amax = 0);
//   q = satfinite-rne_e4m3(fl(x / s)).
// x is a bf16 or fp16 activation, or silu(gate) * up of a bf16 gate_up row,
// which stays in fp32 up to its one rounding to e4m3 (a bf16 step in between
// would move a block's scale by up to 2^-8 whenever it moved its maximum).
//
// A block is 16 chunks of 8 elements: a half-warp holds it in registers, one
// 16-byte load (two for gate and up) per lane, and its maximum is a 4-step
// butterfly over the half-warp. No row-wide reduction exists, so a row is cut
// into as many half-warps as it has blocks and one token fills several SMs.
// Bound by HBM: 2 (or 4) bytes read and 1 + 4/128 written per element. Each
// half-warp takes kUnits consecutive blocks of a row (one index division per
// kUnits blocks) and loads them all before it reduces the first.
#include "common.cuh"
#include "launch.h"

namespace w4 {
namespace {

constexpr int kBlk8 = 16;       // 8-element chunks per block of 128 columns
constexpr int kThreads = 256;

// e4m3 codes of fl(x / s) for 8 fp32 values (the bracket of quant_e4m3_chunk
// holds for any finite fp32 x).
W4_DEV uint2 quant_e4m3_f32(const float (&x)[8], const QuotientBracket& b) {
  uint32_t p[4];
  uint32_t diff = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float l0, l1, h0, h1;
    mul2(l0, l1, x[2 * i], x[2 * i + 1], b.rlo);
    mul2(h0, h1, x[2 * i], x[2 * i + 1], b.rhi);
    p[i] = e4m3x2_rn(l0, l1);
    diff |= p[i] ^ e4m3x2_rn(h0, h1);
  }
  if (diff != 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = e4m3x2_rn(__fdiv_rn(x[2 * i], b.s), __fdiv_rn(x[2 * i + 1], b.s));
  }
  return make_uint2(prmt(p[0], p[1], 0x5410u), prmt(p[2], p[3], 0x5410u));
}

// silu(g) = g / (1 + e^-g) with the one exponential t = e^-|g| in (0, 1]: the
// denominator stays in [1, 2], inside the fast divide's range for every g.
W4_DEV float silu_f32(float g) {
  const float t = __expf(-fabsf(g));
  return __fdividef(g >= 0.f ? g : g * t, 1.f + t);
}

// x [*, K8 chunks], or with kSilu [*, 2 K8]; row r of the output comes from row
// gather[r] (gather may be null: row r). An id outside [0, T) gives a zero row
// with scales 1 and W4_ERR_SHAPE in the status word. KU = ceil(KB / kUnits).
template <bool kF16, bool kSilu, int kUnits>
__global__ void __launch_bounds__(kThreads) quant_block_kernel(const uint4* __restrict__ x, int64_t items, int K8,
                                                               int KB, int KU, uint2* __restrict__ q,
                                                               float* __restrict__ scale,
                                                               const int32_t* __restrict__ gather, int64_t T,
                                                               unsigned int* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int l = threadIdx.x & (kBlk8 - 1);
  const int64_t it = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / kBlk8;
  const bool live = it < items;                 // dead half-warps still take part in the shuffles
  const int64_t row = live ? it / KU : 0;
  const int b0 = live ? static_cast<int>(it - row * KU) * kUnits : KB;
  int64_t src = row;
  bool bad = false;
  if (gather != nullptr && live) {
    src = gather[row];
    bad = src < 0 || src >= T;
  }
  const uint4* xr = x + src * static_cast<int64_t>(kSilu ? 2 * K8 : K8);
  uint4 v[kUnits], u[kSilu ? kUnits : 1];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int c = (b0 + i) * kBlk8 + l;
    const bool in = c < K8 && live && !bad;
    v[i] = in ? ld_stream_v4(xr + c) : make_uint4(0, 0, 0, 0);
    if constexpr (kSilu) u[i] = in ? ld_stream_v4(xr + K8 + c) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int b = b0 + i, c = b * kBlk8 + l;
    uint2 code;
    float s;
    if constexpr (kSilu) {
      const uint32_t g[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      float a[8], m = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[2 * j] = silu_f32(bf16_lo(g[j])) * bf16_lo(w[j]);
        a[2 * j + 1] = silu_f32(bf16_hi(g[j])) * bf16_hi(w[j]);
        m = fmaxf(m, fmaxf(fabsf(a[2 * j]), fabsf(a[2 * j + 1])));
      }
      s = block_scale(half_warp_max(m));
      code = quant_e4m3_f32(a, quotient_bracket(s));
    } else {
      quant_block_half_warp<kF16>(v[i], code, s);
    }
    if (c < K8 && live) q[row * K8 + c] = code;
    if (l == 0 && live && b < KB) scale[row * KB + b] = s;
  }
  if (bad && l == 0) report(status, W4_ERR_SHAPE);
}

template <bool kF16, bool kSilu, int kUnits>
cudaError_t launch(const void* x, int64_t M, int64_t K, const int32_t* gather, int64_t T, void* q, float* scale,
                   unsigned int* status, cudaStream_t s) {
  const int K8 = static_cast<int>(K / 8), KB = static_cast<int>((K + 127) / 128), KU = (KB + kUnits - 1) / kUnits;
  const int64_t items = M * KU;
  const int64_t blocks = (items * kBlk8 + kThreads - 1) / kThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  quant_block_kernel<kF16, kSilu, kUnits><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
      static_cast<const uint4*>(x), items, K8, KB, KU, static_cast<uint2*>(q), scale, gather, T, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_block(const void* x, bool f16, bool silu, int64_t M, int64_t K, const int32_t* gather,
                               int64_t T, void* q, float* scale, unsigned int* status, cudaStream_t s) {
  if (silu) return launch<false, true, 2>(x, M, K, gather, T, q, scale, status, s);
  return f16 ? launch<true, false, 4>(x, M, K, gather, T, q, scale, status, s)
             : launch<false, false, 4>(x, M, K, gather, T, q, scale, status, s);
}

}  // namespace w4
