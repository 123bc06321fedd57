// Activation quantization for the fp8 block-scaled layer: e4m3 codes with one
// fp32 scale per row and 128 columns.
//
// Per row and block b of 128 columns (the last one may be shorter):
//   amax = max |x|;  s = amax / 448 (IEEE fp32 divide; s = 1 where that is 0);
//   q = satfinite-rne_e4m3(fl(x / s)).
// x is a bf16 or fp16 activation, or silu(gate) * up of a bf16 gate_up row,
// which stays in fp32 up to its one rounding to e4m3 (a bf16 step in between
// would move a block's scale by up to 2^-8 whenever it moved its maximum). The gate is
// expf and a division that comes out as IEEE's but for rare last bits, and so does
// x / s: of 369 M codes of normal gates and ups none differed from the formula's in IEEE
// fp32 steps. Cheaper gates took 13 and 28% less time than the first form of these and made
// codes wrong by fp64 where IEEE steps were right (and about as many the other way around):
// ex2.approx in place of expf 48 of the 369 M, the quotient g r unrefined as well 151.
//
// A block is 16 chunks of 8 elements: a half-warp holds it in registers, one
// 16-byte load (two for gate and up) per lane. No row-wide reduction exists, so a
// row is cut into as many half-warps as it has groups of kUnits blocks, and one
// token fills several SMs. Bound by HBM (2 or 4 bytes read and 1 + 4/128 written
// per element) once the instructions are few enough: the kUnits maxima of a
// half-warp are reduced together, lanes trading one half of their values for the
// other at each of the first steps, which leaves the maximum of unit l % kUnits
// in lane l; each lane then divides once, for its unit, and the scales come back
// by shuffles. 32768 x 2048 bf16 takes 33.2 us a call (0.90 of copy bandwidth), 4097 x 4096
// 9.5 (0.79, of which 2 are the launch and the last wave); 32768 x 1408 silu 45.8 on normal
// gates and ups, 48.7 with a column in a hundred 20 times larger, bound by instruction issue
// (26 instructions an element).
#include "common.cuh"
#include "launch.h"

namespace w4 {
namespace {

constexpr int kBlk8 = 16;       // 8-element chunks per block of 128 columns
// Blocks of 128 columns a half-warp: with two, 32768 x 1408 silu took 53.5 us against 49.8,
// and 32768 x 2048 bf16 42.0 against 34.5 (blocks of 256 threads).
constexpr int kUnits = 4;
constexpr int kThreads = 128;    // 4097 x 4096 9.8 us against 10.1 in blocks of 256 threads
constexpr unsigned kFull = 0xFFFFFFFFu;

// -silu(g) * u of any gate. Far below zero the denominator overflows long before the
// product with a large u vanishes: there silu(g) = g exp(g), whose exponential is taken in
// four factors, two on either side of u, so that an underflow before the end is one of the
// product itself (gates down to -180 at the largest u; within 8 ulp). A gate of +inf
// follows the formula, -inf gives NaN.
W4_DEV float neg_silu_mul(float g, float u) {
  if (g < -64.f) {
    const float h = expf(0.25f * g);
    return -(g * h * h * u * h * h);
  }
  return -(__fdiv_rn(g, 1.f + expf(-g)) * u);
}

// x [*, K8 chunks], or with kSilu [*, 2 K8]; row r of the output comes from row
// gather[r] (gather may be null: row r). An id outside [0, T) gives a zero row
// with scales 1 and W4_ERR_SHAPE in the status word. KU = ceil(KB / kUnits). late:
// the next kernel starts only when every kernel before this one is done.
// At least seven silu blocks an SM: 45.8 us at 32768 x 1408 (six 47.0, eight 45.5 in the
// same run, by what the registers leave in flight).
template <bool kF16, bool kSilu>
__global__ void __launch_bounds__(kThreads, kSilu ? 7 : 1) quant_block_kernel(const uint4* x, uint32_t items, int K8,
                                                               int KB, uint32_t KU, uint2* __restrict__ q,
                                                               float* __restrict__ scale,
                                                               const int32_t* gather, int64_t T,
                                                               bool late, unsigned int* status) {
  if (!late) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int l = threadIdx.x & (kBlk8 - 1);
  const uint32_t it = blockIdx.x * (kThreads / kBlk8) + threadIdx.x / kBlk8;
  const bool live = it < items;                 // dead half-warps still take part in the shuffles
  const uint32_t row = it / KU;
  const int b0 = static_cast<int>(it - row * KU) * kUnits;
  int64_t src = row;
  bool bad = false;
  // The kernel before may still be running when this one starts (see launch): x and
  // the row ids may come from it, and it may still be reading q.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (late) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (gather != nullptr && live) {
    src = __ldcg(gather + row);
    bad = src < 0 || src >= T;
  }
  const int c0 = live ? b0 * kBlk8 + l : K8;
  const uint4* xr = x + src * static_cast<int64_t>(kSilu ? 2 * K8 : K8);
  uint4 v[kUnits], u[kSilu ? kUnits : 1];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int c = c0 + i * kBlk8;
    const bool in = c < K8 && !bad;
    v[i] = in ? ld_once_v4(xr + c) : make_uint4(0, 0, 0, 0);
    if constexpr (kSilu) u[i] = in ? ld_once_v4(xr + K8 + c) : make_uint4(0, 0, 0, 0);
  }
  float m[kUnits], a[kSilu ? kUnits : 1][8];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if constexpr (kSilu) {
      const uint32_t g[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      m[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        neg_silu4_mul2(g[j], w[j], a[i][2 * j], a[i][2 * j + 1]);
        m[i] = max_of<true>(m[i], max_of<true>(fabsf(a[i][2 * j]), fabsf(a[i][2 * j + 1])));
      }
    } else {
      m[i] = chunk_max<kF16>(v[i]);
    }
  }
  uint2* qr = q + static_cast<size_t>(row) * K8;
  float* sr = scale + static_cast<size_t>(row) * KB + b0;
  // lane l holds scale and reciprocal of block b0 + l % kUnits (silu: of four times its products)
  const float amax = unit_max<kSilu>(m);
  const float s_mine = kSilu && amax == 0.f ? 4.f : block_scale(amax), r_mine = __frcp_rn(s_mine);
  if (l < kUnits && live && b0 + l < KB) sr[l] = kSilu ? 0.25f * s_mine : s_mine;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const float s = __shfl_sync(kFull, s_mine, i, kBlk8), r = __shfl_sync(kFull, r_mine, i, kBlk8);
    const int c = c0 + i * kBlk8;
    if (c < K8) {
      if constexpr (kSilu) {
        qr[c] = quant_e4m3_refined<1, true>(a[i], s, r);
      } else {
        float f[8];
        chunk_f32<kF16>(v[i], f);
        qr[c] = quant_e4m3_block(f, s, r);
      }
    }
  }
  if constexpr (kSilu) {
    // A block whose scale is out of range (far or infinite gates, NaN, tiny or huge
    // products) is rare: it is read, computed and written once more. Its branch stands
    // apart, so that the arithmetic above overlaps as if it were not there (far gates
    // looked for and mended between products and maximum 48.8 us, before the products 50.3).
    const bool again = !scale_refines(s_mine);
    if (__any_sync(kFull, again)) {
#pragma unroll 1
      for (int i = 0; i < kUnits; ++i) {
        const int c = c0 + i * kBlk8;
        const bool in = c < K8;
        const uint4 gv = in ? ld_once_v4(xr + c) : make_uint4(0, 0, 0, 0);
        const uint4 uv = in ? ld_once_v4(xr + K8 + c) : make_uint4(0, 0, 0, 0);
        const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w}, w[4] = {uv.x, uv.y, uv.z, uv.w};
        float f[8], fm = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = neg_silu_mul(bf16_lo(g[j]), bf16_lo(w[j]));
          f[2 * j + 1] = neg_silu_mul(bf16_hi(g[j]), bf16_hi(w[j]));
          fm = fmaxf(fm, fmaxf(fabsf(f[2 * j]), fabsf(f[2 * j + 1])));
        }
#pragma unroll
        for (int o = kBlk8 / 2; o > 0; o >>= 1) fm = fmaxf(fm, __shfl_xor_sync(kFull, fm, o));
        if (__shfl_sync(kFull, again, i, kBlk8) && in) {
          const float s = block_scale_f32(fm);
          qr[c] = quant_e4m3_block<1, true>(f, s, __frcp_rn(s));
          if (l == 0) sr[i] = s;
        }
      }
    }
  }
  if (bad && l == 0) report(status, W4_ERR_SHAPE);
}

template <bool kF16, bool kSilu>
cudaError_t launch(const void* x, int64_t M, int64_t K, const int32_t* gather, int64_t T, bool late, void* q,
                   float* scale, unsigned int* status, cudaStream_t s) {
  const int K8 = static_cast<int>(K / 8), KB = static_cast<int>((K + 127) / 128), KU = (KB + kUnits - 1) / kUnits;
  const int64_t items = M * KU;
  const int64_t blocks = (items * kBlk8 + kThreads - 1) / kThreads;
  PdlLaunch pl(static_cast<unsigned>(blocks), kThreads, 0, s);
  return cudaLaunchKernelEx(&pl.cfg, quant_block_kernel<kF16, kSilu>, static_cast<const uint4*>(x),
                            static_cast<uint32_t>(items), K8, KB, static_cast<uint32_t>(KU), static_cast<uint2*>(q),
                            scale, gather, T, late, status);
}

// Quantized rows copied to their places among the expert-sorted rows: row r of
// (dst, dst_scale) is row gather[r] of (src, src_scale). A warp per row. The next
// kernel starts only when every kernel before this one is done.
__global__ void __launch_bounds__(kThreads) gather_rows_kernel(const uint4* src,
                                                               const float* src_scale, int64_t T, int K16,
                                                               int KB, const int32_t* gather, int64_t R,
                                                               uint4* __restrict__ dst, float* __restrict__ dst_scale,
                                                               unsigned int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // src comes from the kernel before
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (r >= R) return;
  const int64_t t = __ldcg(gather + r);
  uint4* d = dst + r * K16;
  if (t < 0 || t >= T) {
    for (int i = lane; i < K16; i += 32) d[i] = make_uint4(0, 0, 0, 0);
    for (int i = lane; i < KB; i += 32) dst_scale[r * KB + i] = 1.f;
    if (lane == 0) report(status, W4_ERR_SHAPE);
    return;
  }
  const uint4* s = src + t * K16;
  for (int i0 = 0; i0 < K16; i0 += 128) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 32 * j + lane;
      if (i < K16) v[j] = ld_cg_v4(s + i);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 32 * j + lane;
      if (i < K16) d[i] = v[j];
    }
  }
  for (int i = lane; i < KB; i += 32) dst_scale[r * KB + i] = __ldcg(src_scale + t * KB + i);
}

}  // namespace

bool quant_block_fits(int64_t M, int64_t K) {
  const int64_t per_row = (K + 511) / 512;   // half-warps
  return M <= INT32_MAX / per_row;
}

cudaError_t launch_quant_block(const void* x, bool f16, bool silu, int64_t M, int64_t K, const int32_t* gather,
                               int64_t T, bool late, void* q, float* scale, unsigned int* status, cudaStream_t s) {
  if (silu) return launch<false, true>(x, M, K, gather, T, late, q, scale, status, s);
  return f16 ? launch<true, false>(x, M, K, gather, T, late, q, scale, status, s)
             : launch<false, false>(x, M, K, gather, T, late, q, scale, status, s);
}

cudaError_t launch_gather_block_rows(const void* src, const float* src_scale, int64_t T, int64_t K,
                                     const int32_t* gather, int64_t R, void* dst, float* dst_scale,
                                     unsigned int* status, cudaStream_t s) {
  PdlLaunch pl(static_cast<unsigned>((R + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, s);
  return cudaLaunchKernelEx(&pl.cfg, gather_rows_kernel, static_cast<const uint4*>(src), src_scale, T,
                            static_cast<int>(K / 16), static_cast<int>((K + 127) / 128), gather, R,
                            static_cast<uint4*>(dst), dst_scale, status);
}

}  // namespace w4
