// The few-token expert layer on 4-bit floating point weights (mxfp4, nvfp4), on the
// block-scaled tensor cores: routing, then in two kernels
//
//   up:     h = W_gu[e] x_t                         for every chosen (t, e)
//   down:   a = silu(h_gate) h_up;  y_t = bf16( sum_e w_te W_d[e] a_te ).
//
// The chosen experts' weights are nearly all there is to read: they stream through shared
// memory by TMA and are multiplied as they are (tcgen05 kind::mxf4 and mxf4nvf4, weights on
// the MMA's 128 rows), so that no thread ever unpacks one. For that the activations have to
// be 4-bit floats too: a number becomes a sum of kTerms of them, the digits of a balanced
// octal fraction,
//
//   x = 2^e sum_j d_j 8^-j + r,   d_j in -4 .. 3,
//
// as e2m1 codes 0, 0.5, 1, 1.5, 2 and their negatives, whose magnitude bits count the halves, with
// a block scale 2^(e + 1 - 3 j) per digit. e is chosen per block of columns so that the
// largest magnitude lies in [1.713, 3.427) 2^e, which leaves the first digit within its range,
// and |r| <= 2^(e - 13), 2^-13 of that magnitude: a bf16 number down to 2^-6 of it comes out
// exactly. All digits come from one fp32 addition that aligns the number as an integer and
// adds 4 at every digit, and a few bit operations on eight numbers at a time (the conversion
// instruction for e2m1 takes some 16 cycles a warp). Digits are columns of the MMA's other
// operand, and their products are added in fp32. Those of up to 16 tokens are 80 columns; with
// memory as the bound the tensor core has time for them. (e4m3 holds powers of two from 2^-9
// to 2^8: a token's largest value is brought to [2^7, 2^8), and what falls below 2^-17 of it
// is lost.)
//
// up: the stages of 256 columns of all (expert, tile of 64 gate and 64 up rows) form one list,
// of which every CTA takes an equal share; a tile lies in at most kParts shares, and their
// fp32 sums are added by the down kernel. down: a CTA has 128 outputs and every split-th
// chosen expert, builds the activations' terms while the weights before are multiplied, and
// adds the experts' outputs in order; the CTAs of a cluster add theirs by token. Every sum
// has a fixed order. Where an SM holds a CTA of either kernel, the down kernel routes for itself
// and starts its weights while the up kernel still runs; else it takes the up kernel's choice
// (16 tokens: 108 us with a choice of its own, 102 without).
//
// 16 tokens, 64 experts of 2048 x 1408 in nvfp4, 8 chosen (some 57 of them, 280 MB, 41 us at the
// copy rate): 102 us, the up kernel 40 (10 until the digits of x are there, 28 at the rate of
// memory), the down kernel 60, of which the activations' digits are most. 5 tokens, 96 experts
// of 1024 x 704 in mxfp4, 6 chosen: 25 us.
#include <cstring>

#include "common.cuh"
#include "fp4_codes.cuh"
#include "fp4_scales.cuh"
#include "launch.h"
#include "moe_chosen.cuh"
#include "tc.cuh"
#include "tiles.cuh"

namespace w4 {
namespace {

constexpr int kTerms = 5;
constexpr int kParts = 3;                     // shares that a tile of the up kernel can lie in
constexpr int kStage = 128 * kStageBytes;     // 128 weight rows
constexpr int kMaxStages = 6;
constexpr int kRaw = 128 * 32, kRaws = 2;
constexpr int kThreads = 512;
constexpr int kTeamWarps = 4, kTeam = 32 * kTeamWarps;   // of two teams
constexpr int kBlock = 8;                     // tokens of an expert that the down kernel takes at once
constexpr int kMaxI = 2 * 8 * kTeam;         // two items of 8 columns a thread of a team
constexpr int kMaxH = 8192;
constexpr int kTmem = 256, kAccCols = 80;     // two accumulators of up to 80 columns, then scales

struct Params {
  CUtensorMap tm_w;        // up: [2E, I, K/2 bytes] in boxes of 64 rows of two matrices; down: [E, H, K/2 bytes], 128 rows
  CUtensorMap tm_ws;       // the scales alike, 32 bytes a row
  MoeRouteArgs route;      // ids and wts unset
  const uint8_t* w_scale;
  const float* up_global;  // [E] or null
  const float* down_global;
  const uint4* x;          // bf16 [T, H]
  uint4* choice;           // the up kernel's, for the down kernel
  float* part;             // [kParts][rows][2I]: rows of a tile together, 64 gate and 64 up
  uint16_t* y;             // bf16 [T, H]
  int H, I, K, KS, SB;     // of the kernel's weights: columns, stages, scale bytes a row
  int up_ks, up_ctas;      // the up kernel's stages a tile, and CTAs
  int NC, rows, stages, split;
  int token_rows;          // up: rows of the operand a digit, 8 or 16
  int raw;                 // bytes of a slot of scales as they are in memory
  bool tma_scales;
  unsigned int* status;
};

// The up kernel's list of stages: `total` of them, shares for `n` CTAs.
struct Shares {
  unsigned total, n;   // total n fits 32 bits: at most 256 experts, 64 tiles, 32 stages and n = 256
  W4_DEV Shares(const Params& p, int experts) {
    const int tiles = experts * (p.I / 64);
    total = static_cast<unsigned>(tiles * p.up_ks);
    n = static_cast<unsigned>(min(p.up_ctas, 2 * tiles));   // at least half a tile each: a tile lies in three at most
  }
  W4_DEV int start(unsigned c) const { return static_cast<int>(c >= n ? total : total * c / n); }
  W4_DEV int owner(int s) const { return static_cast<int>(((static_cast<unsigned>(s) + 1) * n - 1) / total); }
};

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages], raw_full[kRaws], raw_empty[kRaws];
  uint64_t acc_full[2], acc_empty[2], b_full[2], b_empty[2];
  uint32_t tmem;
  int abort_flag;
};

// Rows of the operand: digit j of token t is row j * rows + t, rows = 8 or 16, so that a token's
// digits have the same place in the swizzle. Where row r's scale lies in its atom: 16 (r % 32)
// + 4 (r / 32).
template <int kRows>
W4_DEV constexpr int scale_at(int j) {
  return (j * kRows & 31) * 16 + (j * kRows >> 5) * 4;
}

// The digits of 8 values of token t, whose block's largest magnitude has bits `bits`: codes, and by
// the block's first lane the scales. b, bs: the stage's operand and scale atoms; i: which 8 of
// its 256 columns.
template <bool kNv, int kRows>
W4_DEV void store_digits(const float (&f)[8], uint32_t bits, uint8_t* b, uint8_t* bs, int t, int i) {
  static_assert(kTerms == 5, "digits of 3 bits in 16");
  const int e = max(static_cast<int>((bits + 0x24A000u) >> 23) - 128, -110);   // the next one for mantissas from 1.713 on
  const float s = __uint_as_float(static_cast<uint32_t>(127 + 12 - e) << 23);   // 8^4 2^-e
  constexpr float kMagic = 12582912.f + 4.f * (1 + 8 + 64 + 512 + 4096);        // 1.5 2^23 and 4 at every digit
  uint32_t y[8], w[4];
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(fmaf(f[k], s, kMagic));    // digit j + 4 at bits 3 (4 - j)
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = prmt(y[k], y[k + 4], 0x5410u);
  uint8_t* code_at = b + t * 128 + (((i >> 2) ^ (t & 7)) << 4) + (i & 3) * 4;
#pragma unroll
  for (int j = 0; j < kTerms; ++j) {
    const int at = 3 * (4 - j);
    // the eight digits, 4 more than they are, in nibbles
    uint32_t z = (w[0] >> at) & 0x00070007u;
#pragma unroll
    for (int k = 1; k < 4; ++k) z = and_or(at > 4 * k ? w[k] >> (at > 4 * k ? at - 4 * k : 0) : w[k] << (at > 4 * k ? 0 : 4 * k - at), 0x00070007u << (4 * k), z);
    // to sign and magnitude: below 4, 4 - z is (z & 3 flipped) + 1
    const uint32_t n = ~z & 0x44444444u, one = n >> 2;
    *reinterpret_cast<uint32_t*>(code_at + j * kRows * 128) = (((z & 0x33333333u) ^ (one | one << 1)) + one) | n << 1;
  }
  // scales 2^(e + 1 - 3 j): e4m3 by its conversion, which gives 0 below 2^-10, where the digit is given up
  uint32_t c[kTerms];
  if constexpr (kNv) {
    const float p0 = __uint_as_float(static_cast<uint32_t>(127 + 1 + e) << 23);
    const uint32_t c01 = e4m3x2_rn(p0, p0 * 0.125f), c23 = e4m3x2_rn(p0 * 0.015625f, p0 * 0.001953125f);
    c[0] = c01, c[1] = c01 >> 8, c[2] = c23, c[3] = c23 >> 8, c[4] = e4m3x2_rn(p0 * 0.000244140625f, 0.f);
  } else {
#pragma unroll
    for (int j = 0; j < kTerms; ++j) c[j] = static_cast<uint32_t>(127 + 1 + e - 3 * j);   // e >= -110
  }
  const int blk = kNv ? i >> 1 : i >> 2;   // of the stage's scales
  if (kNv ? (i & 1) == 0 : (i & 3) == 0) {
    uint8_t* to = bs + (blk >> 2) * 512 + t * 16 + (blk & 3);
#pragma unroll
    for (int j = 0; j < kTerms; ++j) to[scale_at<kRows>(j)] = static_cast<uint8_t>(c[j]);
  }
}

// What brings a maximum (magnitude bits) to [2^7, 2^8), and its inverse; NaN for what is not finite.
W4_DEV float norm_of(uint32_t bits) {
  const int e = min(max(static_cast<int>(bits >> 23), 8), 254);
  return __uint_as_float(static_cast<uint32_t>(min(261 - e, 254)) << 23);   // 2^(7 - (e - 127))
}
W4_DEV float inverse_norm_of(uint32_t bits) {
  if (bits >= kInfBits) return __uint_as_float(0x7FC00000u);
  return __fdiv_rn(1.f, norm_of(bits));
}

// Warps that bring weights in: both kernels walk the same way over (expert, first row, stages
// k0 .. k1) that next() gives.
W4_DEV float silu_mul(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }

template <class Next>
W4_DEV void load_weights(const Params& p, Bars& bar, uint8_t* ring, Next next, bool late) {
  // weights are read once, and 200 MB of them would push the kernels' own instructions out of L2
  const uint64_t policy = tc::evict_first_policy();
  int st = 0, ph = 1, mat, row, k0, k1;
  bool ok = true, waited = !late;
  while (ok && next(mat, row, k0, k1))
    for (int ks = k0; ks < k1; ++ks) {
      if (!waited && ph == 0) {   // the ring is full, and is emptied only after the kernel before
        grid_dependency_wait();
        waited = true;
      }
      if (!(ok = wait_warp(&bar.empty[st], ph, &bar.abort_flag, p.status))) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar.full[st], kStage);
        tc::tma_load_3d_hint(ring + st * kStage, &p.tm_w, &bar.full[st], ks * kStageBytes, row, mat, policy);
      }
      __syncwarp();
      if (++st == p.stages) st = 0, ph ^= 1;
    }
}
// Scales: 32 bytes a row at a time by TMA, or, where a row's are no whole 16 bytes, all of a
// tile's rows as they lie in memory (p.raw bytes a slot).
template <bool kNv, bool kDown, class Next>
W4_DEV void load_scales(const Params& p, Bars& bar, uint8_t* raw, Next next, bool late) {
  constexpr int kSuper = kNv ? 2 : 4;
  const int lane = threadIdx.x & 31;
  int rs = 0, rph = 1, mat, row, k0, k1;
  bool ok = true, waited = !late;
  while (ok && next(mat, row, k0, k1))
    for (int ks = k0; ks < k1; ks = p.tma_scales ? (ks / kSuper + 1) * kSuper : k1) {
      if (!waited && rph == 0) {
        grid_dependency_wait();
        waited = true;
      }
      if (!(ok = wait_warp(&bar.raw_empty[rs], rph, &bar.abort_flag, p.status))) break;
      uint8_t* to = raw + rs * p.raw;
      if (p.tma_scales) {
        if (elect_one()) {
          mbar_arrive_expect_tx(&bar.raw_full[rs], kRaw);
          tc::tma_load_3d(to, &p.tm_ws, &bar.raw_full[rs], ks / kSuper * 32, row, mat);
        }
        __syncwarp();
      } else {
        const uint8_t* src = p.w_scale + (static_cast<size_t>(mat) * (kDown ? p.H : p.I) + row) * p.SB;
        const int half = 64 * p.SB;   // rows come and go in blocks of 64: whole 16 bytes
        const bool two = !kDown || row + 64 < p.H;
        for (int i = lane * 16; i < (two ? 2 * half : half); i += 512)
          tc::copy16_async(smem_addr(to) + i, src + (kDown || i < half ? i : i - half + static_cast<size_t>(p.I) * p.SB));
        tc::copy_async_arrive(&bar.raw_full[rs]);
      }
      if (++rs == kRaws) rs = 0, rph ^= 1;
    }
}
template <bool kNv, class Next>
W4_DEV void turn_scales(const Params& p, Bars& bar, const uint8_t* raw, uint8_t* atoms, Next next, bool late) {
  constexpr int kWords = kNv ? 4 : 2, kSuper = 8 / kWords;
  const int lane = threadIdx.x & 31;
  int st = 0, ph = 1, rs = 0, rph = 0, mat, row, k0, k1;
  bool ok = true, waited = !late;
  while (ok && next(mat, row, k0, k1))
    for (int ks = k0; ks < k1; ++ks) {
      const int sub = ks % kSuper;
      // A ring that comes around holds what was copied after the kernel before: either may be the first to.
      if (!waited && (rph == 1 || ph == 0)) {
        grid_dependency_wait();
        waited = true;
      }
      if ((ks == k0 || (p.tma_scales && sub == 0)) && !(ok = wait_warp(&bar.raw_full[rs], rph, &bar.abort_flag, p.status))) break;
      uint32_t v[4][kWords];
      if (p.tma_scales) {
        load_scale_words<kNv>(raw + rs * p.raw + lane * 32 + sub * kWords * 4, 4, v);
      } else {   // rows of an even number of bytes; past their ends the next rows', which meet no column
        const uint16_t* f = reinterpret_cast<const uint16_t*>(raw + rs * p.raw + lane * p.SB + ks * kWords * 4);
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int j = 0; j < kWords; ++j) v[b][j] = f[b * 16 * p.SB + 2 * j] | static_cast<uint32_t>(f[b * 16 * p.SB + 2 * j + 1]) << 16;
      }
      if (!(ok = wait_warp(&bar.empty[st], ph, &bar.abort_flag, p.status))) break;
      store_scale_atoms<kNv>(atoms + st * kWords * 512 + lane * 16, 512, v);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.full[st]);
      // the slot goes back once its words have arrived in registers and the fence lies between them and the next copy
      if (ks == k1 - 1 || (p.tma_scales && sub == kSuper - 1)) {
        if (lane == 0) mbar_arrive(&bar.raw_empty[rs]);
        if (++rs == kRaws) rs = 0, rph ^= 1;
      }
      if (++st == p.stages) st = 0, ph ^= 1;
    }
}

// One stage's MMAs: weights of ring slot st on the rows, `cols` columns of operand b.
template <bool kNv>
W4_DEV void issue_stage(const Params& p, uint32_t tmem, int acc, int buf, uint32_t ring, uint32_t atoms, uint32_t b,
                        uint32_t bs, int ks, int cols, bool first) {
  constexpr int kWords = kNv ? 4 : 2, kCols = 4 * kWords;
  const uint32_t sw = tmem + 2 * kAccCols + buf * 2 * kCols, sx = sw + kCols;
  const uint64_t wsd = tc::sdesc_scales(atoms), xsd = tc::sdesc_scales(bs);
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    tc::copy_scales(sw + 4 * i, wsd + 32 * i);
    tc::copy_scales(sx + 4 * i, xsd + 32 * i);
  }
  const uint64_t wd = tc::sdesc_sw128(ring), xd = tc::sdesc_sw128(b);
  const uint32_t idesc = tc::idesc_fp4<kNv>(128, 0) | static_cast<uint32_t>(cols >> 3) << 17;
  const int left = p.K - ks * kStageK;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (64 * j >= left) break;
    const int word = kNv ? j : j >> 1;
    const uint32_t id = idesc | (kNv || !(j & 1) ? 0u : (2u << 29) | (2u << 4));
    tc::mma_fp4<kNv>(tmem + acc * kAccCols, wd + 2 * j, xd + 2 * j, id, sw + 4 * word, sx + 4 * word, !first || j > 0 ? 1u : 0u);
  }
}

// The sum of token t's digits: columns t + `rows` j of the accumulator.
W4_DEV float sum_digits(uint32_t taddr, int t, int rows) {
  float v[kTerms];
#pragma unroll
  for (int j = 0; j < kTerms; ++j) v[j] = tc::tmem_ld1_async(taddr + t + rows * j);
  tc::tmem_wait_ld(v);
  return ((v[0] + v[1]) + (v[2] + v[3])) + v[4];
}

W4_DEV void init_bars(const Params& p, Bars& bar) {
  for (int i = 0; i < p.stages; ++i) {
    mbar_init(&bar.full[i], 2);   // the weights, the transposing warp
    mbar_init(&bar.empty[i], 1);
  }
  for (int i = 0; i < kRaws; ++i) {
    mbar_init(&bar.raw_full[i], p.tma_scales ? 1 : 32);
    mbar_init(&bar.raw_empty[i], 1);
  }
  for (int i = 0; i < 2; ++i) {
    mbar_init(&bar.acc_full[i], 1);
    mbar_init(&bar.acc_empty[i], 4);
    mbar_init(&bar.b_full[i], kTeamWarps);
    mbar_init(&bar.b_empty[i], 1 + 4);
  }
  bar.abort_flag = 0;
  fence_mbar_init();
}

W4_DEV void finish(Bars& bar, int mma_warp) {
  if (*const_cast<volatile int*>(&bar.abort_flag)) {   // let copies and MMAs in flight land before the shared memory goes away
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (static_cast<int>(threadIdx.x >> 5) == mma_warp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(bar.tmem, kTmem);
  }
}

// Shared memory: Bars and Routed, then (1024-byte aligned) the ring, the activations' operand,
// its scale atoms, the weights' scale atoms and scales as they are in memory.
constexpr int kHead = (sizeof(Bars) + sizeof(Routed) + 16 + 1023) / 1024 * 1024;

// Warps 0-3 epilogue, 4 MMA issuer and TMEM owner, 5 weights, 6 their scales, 7 their
// transposition.
template <bool kNv, int kRows>
__global__ void __launch_bounds__(kThreads, 2) up_kernel(const __grid_constant__ Params p) {
  constexpr int kWords = kNv ? 4 : 2;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  Bars& bar = *reinterpret_cast<Bars*>(smem);
  Routed& r = *reinterpret_cast<Routed*>(smem + (sizeof(Bars) + 15) / 16 * 16);
  uint8_t* ring = smem + kHead;
  uint8_t* b = ring + p.stages * kStage;
  uint8_t* bs = b + p.KS * p.NC * 128;
  uint8_t* atoms = bs + p.KS * kWords * 512;
  uint8_t* raw = atoms + p.stages * kWords * 512;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = static_cast<int>(p.route.T);
  if (threadIdx.x == 0) init_bars(p, bar);
  if (warp == 4) tc::tmem_alloc(&bar.tmem, kTmem);
  if (warp == 5 && lane == 0) {
    tc::prefetch_tmap(&p.tm_w);
    if (p.tma_scales) tc::prefetch_tmap(&p.tm_ws);
  }
  route_prepare<kThreads>(r);
  grid_dependency_wait();
  launch_dependents();   // this CTA has its tensor memory, which the next kernels could else take first
  route_all<kThreads>(p.route, r, reinterpret_cast<uint32_t*>(ring), [&](int w) {
    // a token's x in digits, by a warp that routes none where there are
    const int t = T <= 8 ? w - 8 : w;
    if (t < 0 || t >= T) return;
    const uint4* xr = p.x + static_cast<size_t>(t) * (p.H / 8);
    uint32_t m = 0;
#pragma unroll 4
    for (int i = lane; i < p.H / 8; i += 32) {
      const uint4 v = ld_cg_v4(xr + i);
      m = __vmaxu2(__vmaxu2(m, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
      m = __vmaxu2(__vmaxu2(m, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
    }
    m = __reduce_max_sync(kFull, max(m & 0xFFFFu, m >> 16)) << 16;   // as fp32 bits
    if (lane == 0) r.x_scale[t] = inverse_norm_of(m);
    const float norm = norm_of(m);
    uint4 next = lane < p.H / 8 ? ld_cg_v4(xr + lane) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int ks = 0; ks < p.KS; ++ks) {   // a stage, 8 columns a lane, the next one's on their way
      const uint4 v = next;
      const int i = (ks + 1) * 32 + lane;
      next = i < p.H / 8 ? ld_cg_v4(xr + i) : make_uint4(0, 0, 0, 0);
      float f[8];
      chunk_f32<false>(v, f);
      uint32_t bits = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[k] *= norm;
        bits = max(bits, __float_as_uint(f[k]) & 0x7FFFFFFFu);
      }
      bits = max(bits, __shfl_xor_sync(kFull, bits, 1));
      if constexpr (!kNv) bits = max(bits, __shfl_xor_sync(kFull, bits, 2));
      store_digits<kNv, kRows>(f, min(bits, 0x437FFFFFu), b + ks * p.NC * 128, bs + ks * kWords * 512, t, lane);
    }
    tc::fence_proxy_async_smem();
  });
  if (blockIdx.x == 0) keep_choice<kThreads>(r, p.choice);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bar.tmem;
  const Shares shares(p, r.n);
  const int tiles = p.I / 64, s_end = shares.start(blockIdx.x + 1);
  // a role's walk over this CTA's share
  auto walk = [&, s = shares.start(blockIdx.x)](int& mat, int& row, int& k0, int& k1) mutable {
    if (s >= s_end) return false;
    const int tile = s / p.KS, a = tile / tiles;
    k0 = s - tile * p.KS;
    k1 = min(p.KS, k0 + s_end - s);
    s += k1 - k0;
    mat = 2 * r.expert[a];
    row = (tile - a * tiles) * 64;
    return true;
  };

  if (warp == 5) {
    tc::fence_proxy_async_smem();   // the ring held the routing's scratch
    load_weights(p, bar, ring, walk, false);
  } else if (warp == 6) {
    load_scales<kNv, false>(p, bar, raw, walk, false);
  } else if (warp == 7) {
    turn_scales<kNv>(p, bar, raw, atoms, walk, false);
  } else {
    if (warp == 4) {
      int st = 0, ph = 0, ac = 0, aph = 1, buf = 0, mat, row, k0, k1;
      bool ok = true;
      while (ok && walk(mat, row, k0, k1)) {
        if (!(ok = wait_warp(&bar.acc_empty[ac], aph, &bar.abort_flag, p.status))) break;
        for (int ks = k0; ks < k1; ++ks) {
          if (!(ok = wait_warp(&bar.full[st], ph, &bar.abort_flag, p.status))) break;
          tc::fence_after_sync();
          if (elect_one()) {
            issue_stage<kNv>(p, tmem, ac, buf, smem_addr(ring) + st * kStage, smem_addr(atoms) + st * kWords * 512,
                             smem_addr(b) + ks * p.NC * 128, smem_addr(bs) + ks * kWords * 512, ks, p.NC, ks == k0);
            tc::commit(&bar.empty[st]);
            if (ks == k1 - 1) tc::commit(&bar.acc_full[ac]);
          }
          __syncwarp();
          buf ^= 1;
          if (++st == p.stages) st = 0, ph ^= 1;
        }
        if (++ac == 2) ac = 0, aph ^= 1;
      }
    } else if (warp < 4) {
      const int o = 32 * warp + lane;
      int ac = 0, aph = 0, mat, row, k0, k1;
      bool ok = true;
      int s = shares.start(blockIdx.x);
      while (ok && walk(mat, row, k0, k1)) {
        const int tile = s / p.KS, a = tile / tiles, e = mat >> 1;
        s += k1 - k0;
        const int part = static_cast<int>(blockIdx.x) - shares.owner(tile * p.KS);
        const float g = p.up_global != nullptr ? __ldcg(p.up_global + e) : 1.f;
        float* out = p.part + (static_cast<size_t>(part) * p.rows + r.first[a]) * (2 * p.I) + 2 * row + o;
        if (!(ok = wait_warp(&bar.acc_full[ac], aph, &bar.abort_flag, p.status))) break;
        tc::fence_after_sync();
        const uint32_t ta = tmem + (static_cast<uint32_t>(32 * warp) << 16) + ac * kAccCols;
        const int n = r.first[a + 1] - r.first[a];
        for (int i = 0; i < n; ++i) {
          const int t = r.token[r.first[a] + i];
          out[static_cast<size_t>(i) * (2 * p.I)] = sum_digits(ta, t, p.token_rows) * r.x_scale[t] * g;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.acc_empty[ac]);
        if (++ac == 2) ac = 0, aph ^= 1;
      }
    }
  }
  __syncwarp();
  finish(bar, 4);
}

// Warps as in up_kernel, 8-15: activations.
// kTogether: few enough registers for an SM to hold a CTA of the up kernel beside.
template <bool kNv, bool kTogether>
__global__ void __launch_bounds__(kThreads, kTogether ? 2 : 1) down_kernel(const __grid_constant__ Params p) {
  constexpr int kWords = kNv ? 4 : 2;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  Bars& bar = *reinterpret_cast<Bars*>(smem);
  Routed& r = *reinterpret_cast<Routed*>(smem + (sizeof(Bars) + 15) / 16 * 16);
  uint8_t* ring = smem + kHead;
  uint8_t* b = ring + p.stages * kStage;             // two
  uint8_t* bs = b + 2 * p.KS * p.NC * 128;
  uint8_t* atoms = bs + 2 * p.KS * kWords * 512;
  uint8_t* raw = atoms + p.stages * kWords * 512;
  const int T = static_cast<int>(p.route.T);
  float* sums = reinterpret_cast<float*>(raw + kRaws * p.raw);   // [T][128]
  float* b_scale = sums + T * 128;                              // [2][kBlock]
  uint32_t* maxima = reinterpret_cast<uint32_t*>(b_scale + 2 * kBlock);   // [team][2][kTeamWarps]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) init_bars(p, bar);
  if (warp == 4) tc::tmem_alloc(&bar.tmem, kTmem);
  if (warp == 5 && lane == 0) {
    tc::prefetch_tmap(&p.tm_w);
    if (p.tma_scales) tc::prefetch_tmap(&p.tm_ws);
  }
  // The next kernels may come once this CTA has its tensor memory, which they could else take first.
  if constexpr (kTogether) {   // while the up kernel runs, which let this one go when all before it were done: the logits are there
    route_prepare<kThreads>(r);
    launch_dependents();
    route_all<kThreads>(p.route, r, reinterpret_cast<uint32_t*>(ring), [](int) {});
  } else {
    __syncthreads();
    launch_dependents();
    grid_dependency_wait();
    take_choice<kThreads>(r, p.choice);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bar.tmem;
  const int rank = p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int n0 = static_cast<int>(blockIdx.x) / p.split * 128;
  // every split-th chosen expert, its tokens kBlock at a time (the weights once for each)
  auto blocks = [&](int a) { return (r.first[a + 1] - r.first[a] + kBlock - 1) / kBlock; };
  auto walk = [&, a = rank, i = 0](int& mat, int& row, int& k0, int& k1) mutable {
    if (a >= r.n) return false;
    mat = r.expert[a];
    row = n0, k0 = 0, k1 = p.KS;
    if (++i == blocks(a)) i = 0, a += p.split;
    return true;
  };

  if (warp == 5) {
    tc::fence_proxy_async_smem();
    load_weights(p, bar, ring, walk, true);
  } else if (warp == 6) {
    load_scales<kNv, true>(p, bar, raw, walk, true);
  } else if (warp == 7) {
    turn_scales<kNv>(p, bar, raw, atoms, walk, true);
  } else if (warp == 4) {
    grid_dependency_wait();
    int st = 0, ph = 0, ac = 0, aph = 1, bph = 0, buf = 0;
    bool ok = true;
    for (int a = rank, i = 0; ok && a < r.n; ++i == blocks(a) ? i = 0, a += p.split : 0) {
      if (!(ok = wait_warp(&bar.acc_empty[ac], aph, &bar.abort_flag, p.status))) break;
      if (!(ok = wait_warp(&bar.b_full[ac], bph, &bar.abort_flag, p.status))) break;
      const uint32_t bo = smem_addr(b) + ac * p.KS * p.NC * 128, bso = smem_addr(bs) + ac * p.KS * kWords * 512;
      for (int ks = 0; ks < p.KS; ++ks) {
        if (!(ok = wait_warp(&bar.full[st], ph, &bar.abort_flag, p.status))) break;
        tc::fence_after_sync();
        if (elect_one()) {
          issue_stage<kNv>(p, tmem, ac, buf, smem_addr(ring) + st * kStage, smem_addr(atoms) + st * kWords * 512,
                           bo + ks * p.NC * 128, bso + ks * kWords * 512, ks, p.NC, ks == 0);
          tc::commit(&bar.empty[st]);
          if (ks == p.KS - 1) {
            tc::commit(&bar.acc_full[ac]);
            tc::commit(&bar.b_empty[ac]);
          }
        }
        __syncwarp();
        buf ^= 1;
        if (++st == p.stages) st = 0, ph ^= 1;
      }
      if (++ac == 2) ac = 0, aph ^= 1, bph ^= 1;
    }
  } else if (warp >= 8) {
    // Two teams of four warps take the blocks of tokens in turn, each with an operand of its
    // own: silu(gate) * up of a token's row, 8 columns an item, two items a thread, then its digits.
    grid_dependency_wait();
    const Shares shares(p, r.n);
    const int team = (warp - 8) / kTeamWarps, tid = threadIdx.x % kTeam, tiles = p.I / 64, all = p.I / 8;
    uint8_t* bo = b + team * p.KS * p.NC * 128;
    uint8_t* bso = bs + team * p.KS * kWords * 512;
    uint32_t* top_of = maxima + team * 2 * kTeamWarps;
    // sums of gate and up of eight of this thread's columns: the first parts, to which the rest is added
    struct Sums {
      float4 g[2], u[2];
    };
    auto fetch = [&](int row, int k, Sums& v) {
      const int i = tid + kTeam * k;
      const float* h = p.part + static_cast<size_t>(row) * (2 * p.I) + (i >> 3) * 128 + (i & 7) * 8;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v.g[j] = i < all ? __ldcg(reinterpret_cast<const float4*>(h + 4 * j)) : make_float4(0.f, 0.f, 0.f, 0.f);
        v.u[j] = i < all ? __ldcg(reinterpret_cast<const float4*>(h + 64 + 4 * j)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    int ph = 1, turn = 0, count = 0;
    bool ok = true;
    int a = rank, blk = 0;
    auto skip = [&]() {   // to this team's next block
      while (a < r.n && (count & 1) != team) {
        ++count;
        if (++blk == blocks(a)) blk = 0, a += p.split;
      }
    };
    skip();
    // With the registers of a whole SM a token's sums are fetched while the digits of the one before
    // are made (16 tokens, 64 experts of 2048 x 1408, 8 chosen: 126 -> 108 us); with half of them
    // that spills, and the other kernel's CTA fills the time (5 tokens, 96 experts of 1024 x 704,
    // 6 chosen: 24.7 us, 27.4 with it).
    constexpr bool kAhead = !kTogether;
    Sums v[2];
    if (kAhead && a < r.n) fetch(r.first[a] + blk * kBlock, 0, v[0]), fetch(r.first[a] + blk * kBlock, 1, v[1]);
    while (a < r.n) {
      const int first = r.first[a] + blk * kBlock, n = min(r.first[a + 1] - first, kBlock);
      int parts[2];   // the other parts of this thread's columns
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int s = (a * tiles + ((tid + kTeam * k) >> 3)) * p.up_ks;
        parts[k] = tid + kTeam * k < all ? shares.owner(s + p.up_ks - 1) - shares.owner(s) : 0;
      }
      ++count;
      if (++blk == blocks(a)) blk = 0, a += p.split;
      skip();
      const int after = a < r.n ? r.first[a] + blk * kBlock : -1;   // first row of the block after this one
      for (int t = 0; t < n; ++t) {
        float f[2][8];
        uint32_t bits[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = tid + kTeam * k;
          Sums& c = v[kAhead ? k : 0];
          if (!kAhead) fetch(first + t, k, c);
          const float* h = p.part + static_cast<size_t>(first + t) * (2 * p.I) + (i >> 3) * 128 + (i & 7) * 8;
          for (int q = parts[k]; q > 0; --q) {
            h += static_cast<size_t>(p.rows) * (2 * p.I);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 g = __ldcg(reinterpret_cast<const float4*>(h + 4 * j)), u = __ldcg(reinterpret_cast<const float4*>(h + 64 + 4 * j));
              c.g[j].x += g.x, c.g[j].y += g.y, c.g[j].z += g.z, c.g[j].w += g.w;
              c.u[j].x += u.x, c.u[j].y += u.y, c.u[j].z += u.z, c.u[j].w += u.w;
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float* to = f[k] + 4 * j;
            to[0] = silu_mul(c.g[j].x, c.u[j].x), to[1] = silu_mul(c.g[j].y, c.u[j].y);
            to[2] = silu_mul(c.g[j].z, c.u[j].z), to[3] = silu_mul(c.g[j].w, c.u[j].w);
#pragma unroll
            for (int e = 0; e < 4; ++e) bits[k] = max(bits[k], __float_as_uint(to[e]) & 0x7FFFFFFFu);
          }
        }
        const int next = t + 1 < n ? first + t + 1 : after;
        if (kAhead && next >= 0) fetch(next, 0, v[0]), fetch(next, 1, v[1]);
        // the row's largest magnitude
        uint32_t m = __reduce_max_sync(kFull, max(bits[0], bits[1]));
        if (lane == 0) top_of[turn * kTeamWarps + warp % kTeamWarps] = m;
        asm volatile("bar.sync %0, %1;" :: "r"(team + 1), "n"(kTeam) : "memory");
#pragma unroll
        for (int k = 0; k < kTeamWarps; ++k) m = max(m, top_of[turn * kTeamWarps + k]);
        turn ^= 1;
        if (t == 0) {   // the operand is needed from here on; after a time-out the warps go on without waiting, so that they still meet
          ok = ok && wait_warp(&bar.b_empty[team], ph, &bar.abort_flag, p.status);
          ph ^= 1;
        }
        if (tid == 0) b_scale[team * kBlock + t] = inverse_norm_of(m);
        const float norm = norm_of(m);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = tid + kTeam * k;
          uint32_t top = __float_as_uint(__uint_as_float(bits[k]) * norm);
          top = max(top, __shfl_xor_sync(kFull, top, 1));
          if constexpr (!kNv) top = max(top, __shfl_xor_sync(kFull, top, 2));
          if (i < all) {
#pragma unroll
            for (int c = 0; c < 8; ++c) f[k][c] *= norm;
            store_digits<kNv, kBlock>(f[k], min(top, 0x437FFFFFu), bo + (i >> 5) * p.NC * 128, bso + (i >> 5) * kWords * 512, t, i & 31);
          }
        }
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.b_full[team]);
    }
  } else {
    const int o = 32 * warp + lane;
    for (int t = 0; t < T; ++t) sums[t * 128 + o] = 0.f;   // this thread's outputs
    grid_dependency_wait();
    int ac = 0, aph = 0;
    bool ok = true;
    for (int a = rank, blk = 0; ok && a < r.n; ++blk == blocks(a) ? blk = 0, a += p.split : 0) {
      const float g = p.down_global != nullptr ? __ldcg(p.down_global + r.expert[a]) : 1.f;
      if (!(ok = wait_warp(&bar.acc_full[ac], aph, &bar.abort_flag, p.status))) break;
      tc::fence_after_sync();
      const uint32_t ta = tmem + (static_cast<uint32_t>(32 * warp) << 16) + ac * kAccCols;
      const int first = r.first[a] + blk * kBlock, n = min(r.first[a + 1] - first, kBlock);
      for (int i = 0; i < n; ++i) {
        float& at = sums[r.token[first + i] * 128 + o];
        at = fmaf(sum_digits(ta, i, kBlock) * b_scale[ac * kBlock + i], g * r.weight[first + i], at);
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.acc_empty[ac]);
        mbar_arrive(&bar.b_empty[ac]);
      }
      if (++ac == 2) ac = 0, aph ^= 1;
    }
  }
  __syncwarp();
  __syncthreads();
  if (p.split > 1) {
    cluster_arrive();
    cluster_wait();
  }
  // tokens rank, rank + split, ...: a warp a token, four outputs a lane, the CTAs in order
  for (int t = rank + warp * p.split; t < T; t += kThreads / 32 * p.split) {
    const uint32_t at = smem_addr(sums + t * 128 + 4 * lane);
    float4 v[kMaxSplit];
#pragma unroll
    for (int k = 0; k < kMaxSplit; ++k)
      if (k < p.split) v[k] = p.split > 1 ? ld_cluster_f32x4(at, k) : *reinterpret_cast<const float4*>(sums + t * 128 + 4 * lane);
    float4 s = v[0];
#pragma unroll
    for (int k = 1; k < kMaxSplit; ++k)
      if (k < p.split) s.x += v[k].x, s.y += v[k].y, s.z += v[k].z, s.w += v[k].w;
    if (n0 + 4 * lane < p.H)
      *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(t) * p.H + n0 + 4 * lane) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
  if (p.split > 1) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  finish(bar, 4);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// A slot of scales: 32 bytes of 128 rows, or all of theirs and what a read past the last row's end may touch.
int raw_bytes(const MoeDecodeArgs& a, bool down) {
  const int64_t SB = (down ? a.I : a.H) / (a.format == W4_FMT_NVFP4 ? 16 : 32);
  return SB % 16 == 0 ? kRaw : static_cast<int>((128 * SB + 32 + 127) / 128 * 128);
}
// Columns of a stage's operand: kTerms times 8 or 16 rows, in whole 16.
int columns(int64_t T) { return T <= 8 ? 48 : 80; }
int64_t smem_bytes(const MoeDecodeArgs& a, bool down, int stages) {
  const int words = a.format == W4_FMT_NVFP4 ? 4 : 2;
  const int64_t ks = ((down ? a.I : a.H) + kStageK - 1) / kStageK, T = down ? kBlock : a.route.T;
  return 1024 + kHead + static_cast<int64_t>(stages) * (kStage + words * 512) + (down ? 2 : 1) * ks * (columns(T) * 128 + words * 512) +
         kRaws * raw_bytes(a, down) + (down ? a.route.T * 512 + 2 * kBlock * 4 + 4 * kTeamWarps * 4 : 0);
}

template <bool kNv>
cudaError_t run(const MoeDecodeArgs& a, bool down, cudaStream_t s) {
  Params p;
  memset(&p, 0, sizeof(p));
  p.route = a.route;
  p.K = static_cast<int>(down ? a.I : a.H);
  p.H = static_cast<int>(a.H);
  p.I = static_cast<int>(a.I);
  p.KS = (p.K + kStageK - 1) / kStageK;
  p.SB = p.K / static_cast<int>(fp4_block(kNv));
  p.up_ks = static_cast<int>((a.H + kStageK - 1) / kStageK);
  p.up_ctas = current_sm_count() < 256 ? current_sm_count() : 256;
  p.w_scale = static_cast<const uint8_t*>(down ? a.down_scale : a.gate_up_scale);
  p.up_global = a.gate_up_global;
  p.down_global = a.down_global;
  p.x = static_cast<const uint4*>(a.x);
  p.choice = static_cast<uint4*>(a.workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kMoeChoiceBytes);
  p.y = static_cast<uint16_t*>(a.y);
  p.NC = columns(down ? kBlock : a.route.T);
  p.token_rows = a.route.T <= 8 ? 8 : 16;
  p.rows = static_cast<int>(a.route.T) * a.route.k;
  p.tma_scales = p.SB % 16 == 0;
  p.raw = raw_bytes(a, down);
  p.status = a.status;
  const void* w = down ? a.down : a.gate_up;
  const int64_t rows = down ? a.H : a.I, mats = down ? a.route.E : 2 * a.route.E;
  const int box = down ? 128 : 64, pair = down ? 1 : 2;
  cudaError_t e = encode(&p.tm_w, w, p.K / 2, rows, mats, box, pair);
  if (e == cudaSuccess && p.tma_scales) e = encode(&p.tm_ws, p.w_scale, p.SB, rows, mats, box, pair, 32);
  if (e != cudaSuccess) return e;
  // Where both kernels fit an SM together, the second one's first stages arrive while the
  // first still runs: the up kernel gets what the down kernel leaves with three stages.
  const int64_t both = 233472 - 2 * 1024;
  int up = kMaxStages, dn = kMaxStages;
  const bool together = smem_bytes(a, false, 3) + smem_bytes(a, true, 3) <= both;
  if (together) {
    while (smem_bytes(a, false, up) + smem_bytes(a, true, 3) > both) --up;
    while (smem_bytes(a, false, up) + smem_bytes(a, true, dn) > both) --dn;
  } else {
    while (smem_bytes(a, false, up) > 232448) --up;
    while (smem_bytes(a, true, dn) > 232448) --dn;
  }
  p.stages = down ? dn : up;
  p.split = 1;
  const int smem = static_cast<int>(smem_bytes(a, down, p.stages));
  if (!down) return a.route.T <= 8 ? start<up_kernel<kNv, 8>>(p, p.up_ctas, kThreads, smem, 1, s, 232448) : start<up_kernel<kNv, 16>>(p, p.up_ctas, kThreads, smem, 1, s, 232448);
  const int64_t slices = (a.H + 127) / 128;
  for (int n = kMaxSplit; n > 1 && p.split == 1; n /= 2)
    if (slices * n <= current_sm_count() && n <= p.rows) p.split = n;
  return together ? start<down_kernel<kNv, true>>(p, slices * p.split, kThreads, smem, p.split, s, 232448)
                  : start<down_kernel<kNv, false>>(p, slices * p.split, kThreads, smem, p.split, s, 232448);
}

}  // namespace

size_t moe_decode_fp4_workspace_bytes(int64_t T, int64_t k, int64_t I) {
  return kMoeChoiceBytes + static_cast<size_t>(kParts) * static_cast<size_t>(T * k) * static_cast<size_t>(2 * I) * sizeof(float);
}

// Room for three stages beside the activations.
bool moe_decode_fp4_fits(const MoeDecodeArgs& a) {
  if (a.format == W4_FMT_INT4 || a.I > kMaxI || a.H > kMaxH) return false;
  return smem_bytes(a, false, 3) <= 232448 && smem_bytes(a, true, 3) <= 232448;
}

cudaError_t launch_moe_decode_fp4(const MoeDecodeArgs& a, cudaStream_t s) {
  const bool nv = a.format == W4_FMT_NVFP4;
  const cudaError_t e = nv ? run<true>(a, false, s) : run<false>(a, false, s);
  if (e != cudaSuccess) return e;
  return nv ? run<true>(a, true, s) : run<false>(a, true, s);
}

}  // namespace w4
