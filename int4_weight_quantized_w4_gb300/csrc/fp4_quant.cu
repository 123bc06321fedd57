// Microscaled 4-bit floats: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives) with a scale per block of columns of a row.
//
//   mxfp4: blocks of 32; scale 2^e, e = clamp(floor(log2 amax) - 2, -127, 127), kept
//          as e + 127 (e8m0); q = rne_e2m1(x 2^-e), held to +-6.
//   nvfp4: blocks of 16 and an fp32 scale g of the whole tensor; s = rne_e4m3(fl(fl(amax
//          / 6) / g)), held to 448; d = fl(s g); q = rne_e2m1(fl(x / d)), held to +-6 (0
//          where d is 0).
//
// x is a bf16 or fp16 activation, or silu(gate) * up of a bf16 gate_up row, in fp32 steps:
// fl(fl(g / fl(1 + expf(-g))) up), the quotient within an ulp of IEEE's. A block that holds a NaN or an infinity gets
// a NaN scale, so that it shows in whatever is computed from it.
//
// K is a multiple of the block, so blocks of a row-major matrix follow one another
// whatever the rows, and a thread takes 16 consecutive elements: an nvfp4 block, or
// half an mxfp4 block whose other half is the neighbour lane's. No row-wide step
// exists. Bound by HBM: 2 or 4 bytes read and 1/2 + 1/16 (1/32) written an element.
#include "common.cuh"
#include "fp4_codes.cuh"
#include "launch.h"

namespace w4 {
namespace {

constexpr int kThreads = 128;
constexpr unsigned kFull = 0xFFFFFFFFu;

// Item i: 16 elements of the output; a thread has kItems of them, whose loads are in flight
// together. kSilu: columns c and K + c of the row's 2 K. gather (may be null): source row of each output
// row; an id outside [0, T) gives a zero row and W4_ERR_SHAPE in the status word. K16 = K / 16. wide: x
// is 32-byte aligned. signals: the next kernel may start once every kernel before this one is done; else when
// this one is, which may have written weights.
template <bool kNv, bool kF16, bool kSilu, int kItems>
__global__ void __launch_bounds__(kThreads) quant_fp4_kernel(const uint4* x, int64_t items, uint32_t K16,
                                                             const float* global, const int32_t* gather, int64_t T,
                                                             bool signals, bool wide, uint2* __restrict__ q,
                                                             uint8_t* __restrict__ scale, unsigned int* status) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kItems) + threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // x may come from the kernel before, which may still read q
  if (signals) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint4 v[kItems][2], u[kItems][2];   // u: kSilu
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    const int64_t i = i0 + n * kThreads;
    v[n][0] = v[n][1] = u[n][0] = u[n][1] = make_uint4(0, 0, 0, 0);
    if (i >= items) continue;
    int64_t at = i;
    if (kSilu || gather != nullptr) {
      const int64_t row = i / K16;
      const uint32_t c = static_cast<uint32_t>(i - row * K16);
      int64_t src = row;
      if (gather != nullptr) {
        src = __ldcg(gather + row);
        if (src < 0 || src >= T) {
          if (c == 0) report(status, W4_ERR_SHAPE);
          continue;
        }
      }
      at = src * (kSilu ? 2 * K16 : K16) + c;
    }
    load32(x + 2 * at, wide, v[n]);
    if constexpr (kSilu) load32(x + 2 * (at + K16), wide, u[n]);
  }
  const float g = kNv && global != nullptr ? *global : 1.f;
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    const int64_t i = i0 + n * kThreads;
    float f[2][8];
    uint32_t bits = 0;
    if constexpr (kSilu) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t gw[4] = {v[n][h].x, v[n][h].y, v[n][h].z, v[n][h].w}, uw[4] = {u[n][h].x, u[n][h].y, u[n][h].z, u[n][h].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float a0, a1;
          neg_silu4_mul2(gw[j], uw[j], a0, a1);
          mul2(f[h][2 * j], f[h][2 * j + 1], a0, a1, -0.25f);
          bits = max(bits, max(__float_as_uint(f[h][2 * j]) & 0x7FFFFFFFu, __float_as_uint(f[h][2 * j + 1]) & 0x7FFFFFFFu));
        }
      }
      // far or infinite gates and products beyond a quarter of the largest number show as
      // infinities or NaN there; products below 2^-120 have lost bits: by the formula's steps
      if (bits >= kInfBits || bits < (7u << 23)) {
        bits = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float a[8];
          chunk_f32<false>(v[n][h], a);
          chunk_f32<false>(u[n][h], f[h]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f[h][j] *= __fdiv_rn(a[j], 1.f + expf(-a[j]));
            bits = max(bits, __float_as_uint(f[h][j]) & 0x7FFFFFFFu);
          }
        }
      }
    } else {
      bits = widen16<kF16>(v[n], f);
    }
    if constexpr (!kNv) bits = max(bits, __shfl_xor_sync(kFull, bits, 1));
    if (i >= items) continue;   // an odd half of the last warp took part in the shuffle
    uint2 code;
    const uint32_t s = block_codes<kNv>(f, bits, g, code);
    q[i] = code;
    if constexpr (kNv)
      scale[i] = static_cast<uint8_t>(s);
    else if ((i & 1) == 0)
      scale[i >> 1] = static_cast<uint8_t>(s);
  }
}

// From so many items on a product that starts early takes SMs from the quantizer that it waits for (N 11008, K
// 4096, early / not, nvfp4: 256 rows, 2^16 items, 13.1 / 14.1 us; 1024 32.8 / 32.3, 1536 42.0 / 40.8, 2048, 2^19 items,
// 55.9 / 54.1, 4096 98.7 / 92.6; mxfp4: 256 12.3 / 13.1, 1024 29.1 / 29.2, 2048 49.8 / 49.0, 4096 89.3 / 82.9).
constexpr int64_t kMany = 1 << 19;

template <bool kNv, bool kF16, bool kSilu, int kItems>
cudaError_t launch_items(const QuantFp4Args& a, int64_t items, cudaStream_t s) {
  constexpr int kPer = kThreads * kItems;
  PdlLaunch pl(static_cast<unsigned>((items + kPer - 1) / kPer), kThreads, 0, s);
  return cudaLaunchKernelEx(&pl.cfg, quant_fp4_kernel<kNv, kF16, kSilu, kItems>, static_cast<const uint4*>(a.x), items,
                            static_cast<uint32_t>(a.K / 16), a.global, a.gather, a.T, a.signals && items < kMany, (reinterpret_cast<uintptr_t>(a.x) & 31) == 0, static_cast<uint2*>(a.q),
                            static_cast<uint8_t*>(a.scale), a.status);
}

// Two items a thread where there are many: 14336 x 4096 nvfp4 28.7 -> 26.9 us, mxfp4 22.4 -> 22.0; at 4097
// x 1408, 360,000 items, nvfp4 takes 3.6 us with one and 3.8 with two. silu has two loads a thread already.
template <bool kNv, bool kF16, bool kSilu>
cudaError_t launch(const QuantFp4Args& a, cudaStream_t s) {
  const int64_t items = a.M * (a.K / 16);
  if constexpr (!kSilu)
    if (items >= kMany) return launch_items<kNv, kF16, kSilu, 2>(a, items, s);
  return launch_items<kNv, kF16, kSilu, 1>(a, items, s);
}

// Values of 16 codes: rounded once, from fl(q d) with d = fl(s g), or from q 2^e.
template <bool kNv, bool kF16>
__global__ void __launch_bounds__(kThreads) dequant_fp4_kernel(const uint2* q, const uint8_t* scale,
                                                               const float* global, int64_t items, bool wide,
                                                               uint4* __restrict__ out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (i >= items) return;
  const uint2 c = __ldcg(q + i);
  const uint32_t s8 = __ldcg(scale + (kNv ? i : i >> 1));
  float d;
  if constexpr (kNv) {
    d = half_bits_to_f32(e4m3x2_to_f16x2(s8) & 0xFFFFu) * (global != nullptr ? *global : 1.f);   // from L1: one L2 line for every warp took 36 us in place of 23
  } else {
    d = __uint_as_float(s8 == 0 ? 1u << 22 : s8 == 255 ? 0x7FC00000u : s8 << 23);
  }
  uint4 v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[4], o[4];
    e2m1x8_to_f16(h ? c.y : c.x, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      mul2(lo, hi, half_bits_to_f32(w[j] & 0xFFFFu), half_bits_to_f32(w[j] >> 16), d);
      if constexpr (kF16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[j]) : "f"(hi), "f"(lo));
      else
        o[j] = pack_bf16x2(lo, hi);
    }
    v[h] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (wide) {
    st_v8(out + 2 * i, v[0], v[1]);
  } else {
    out[2 * i] = v[0];
    out[2 * i + 1] = v[1];
  }
}

// Quantized rows copied to their places among the expert-sorted rows: row r of (dst,
// dst_scale) is row gather[r] of (src, src_scale), codes of K16 chunks of 16 bytes and scales
// of SW words. A warp per row.
__global__ void __launch_bounds__(kThreads) gather_fp4_rows_kernel(const uint4* src, const uint32_t* src_scale, int64_t T,
                                                                   int K16, int SW, const int32_t* gather, int64_t R,
                                                                   uint4* __restrict__ dst, uint32_t* __restrict__ dst_scale,
                                                                   unsigned int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // src comes from the kernel before
  if (r >= R) return;
  const int64_t t = __ldcg(gather + r);
  uint4* d = dst + r * K16;
  uint32_t* ds = dst_scale + r * SW;
  if (t < 0 || t >= T) {
    for (int i = lane; i < K16; i += 32) d[i] = make_uint4(0, 0, 0, 0);
    for (int i = lane; i < SW; i += 32) ds[i] = 0;
    if (lane == 0) report(status, W4_ERR_SHAPE);
    return;
  }
  const uint4* s = src + t * K16;
  const uint32_t* ss = src_scale + t * SW;
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
  for (int i = lane; i < SW; i += 32) ds[i] = __ldcg(ss + i);
}

}  // namespace

bool quant_fp4_fits(int64_t M, int64_t K) {
  return M <= static_cast<int64_t>(INT32_MAX) * kThreads / (K / 16);
}

cudaError_t launch_quant_fp4(const QuantFp4Args& a, cudaStream_t s) {
  if (a.silu) return a.nv ? launch<true, false, true>(a, s) : launch<false, false, true>(a, s);
  if (a.f16) return a.nv ? launch<true, true, false>(a, s) : launch<false, true, false>(a, s);
  return a.nv ? launch<true, false, false>(a, s) : launch<false, false, false>(a, s);
}

cudaError_t launch_gather_fp4_rows(const void* src, const void* src_scale, int64_t T, int64_t K, bool nv,
                                   const int32_t* gather, int64_t R, void* dst, void* dst_scale, unsigned int* status,
                                   cudaStream_t s) {
  PdlLaunch pl(static_cast<unsigned>((R + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, s);
  return cudaLaunchKernelEx(&pl.cfg, gather_fp4_rows_kernel, static_cast<const uint4*>(src),
                            static_cast<const uint32_t*>(src_scale), T, static_cast<int>(K / 32),
                            static_cast<int>(K / fp4_block(nv) / 4), gather, R, static_cast<uint4*>(dst),
                            static_cast<uint32_t*>(dst_scale), status);
}

cudaError_t launch_dequant_fp4(const void* q, const void* scale, const float* global, bool nv, bool f16, int64_t M,
                               int64_t K, void* out, cudaStream_t s) {
  const int64_t items = M * (K / 16);
  PdlLaunch pl(static_cast<unsigned>((items + kThreads - 1) / kThreads), kThreads, 0, s);
  auto* kernel = nv ? (f16 ? dequant_fp4_kernel<true, true> : dequant_fp4_kernel<true, false>)
                    : (f16 ? dequant_fp4_kernel<false, true> : dequant_fp4_kernel<false, false>);
  return cudaLaunchKernelEx(&pl.cfg, kernel, static_cast<const uint2*>(q), static_cast<const uint8_t*>(scale), global,
                            items, (reinterpret_cast<uintptr_t>(out) & 31) == 0, static_cast<uint4*>(out));
}

}  // namespace w4
