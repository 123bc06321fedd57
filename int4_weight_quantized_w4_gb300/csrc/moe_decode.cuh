// A whole mixture-of-experts layer for a few tokens, in two kernels: 4-bit weights
// (int4 with fp16 group scales, mxfp4 or nvfp4), 16-bit activations.
//
//   route:  as route.cuh;
//   up:     h = W_gu[e] x_t;  a = silu(h_gate) h_up            for every chosen (t, e)
//   down:   y_t = bf16( sum_e w_te W_d[e] a_te ).
//
// The chosen experts' weights are nearly all there is to read, each weight once: bound by
// HBM. The first kernel routes, in every CTA, and leaves the choice to the second one.
//
// A unit of work is 32 weight rows of one expert: 16 gate rows and their 16 up rows
// (up), or 32 output columns (down). Four warps take a unit together, each a quarter of
// every 512 columns, and add their sums in shared memory; a CTA has four such groups, each
// with a ring of row pieces that TMA keeps full. The products
// are mma.m16n8k16 in fp16 with fp32 sums: at 8 tokens an expert or fewer the tensor
// core idles either way, and what counts is how few instructions turn a 32-bit word of
// weights into operand registers. A word is 8 consecutive columns of a row, and a lane's
// words are its operands as they lie: columns 8 c .. 8 c + 7 of 32 belong to lane c of a
// quad for weights and activations alike, so that no shuffle is needed. int4 codes become
// q - 8 by (q | 1024) - 1032 (exact in fp16, four words of five steps), e2m1 codes by the
// conversion instruction (byte permutations of a table and the sign apart, 15 instructions a word, took
// 129 us for 16 tokens in nvfp4 where this took 103); nvfp4 block scales are multiplied in (six
// mantissa bits, exact), the others scale fp32 sums of their group. A piece's scales come with it where
// rows of them are whole 16 bytes for TMA, else a unit's with its first piece (16 tokens in nvfp4 103 us by the
// piece, 120 by the unit).
//
// Activations are fp16 numbers times a power of two: x_t with its largest magnitude in
// [2^14, 2^15) (a bf16 keeps all its bits down to 2^-29 of that), a_te the same over every
// eight columns, in two halves: fp16 rounds a to 11 bits, and a second number takes the next 11. The
// halves are columns of the product side by side, which costs nothing up to four tokens an expert.
// Those exponents differ along k; a warp brings its columns to the
// largest of them before it multiplies, which takes bits only from what lies below 2^-29 of it.
//
// One token, 64 experts of 2048 x 1408 in int4, 8 chosen (34.6 MB, 5.3 us at the copy rate): 24 us,
// of which 4 go to the choice of experts and 4 to the second kernel's start, most of the rest to
// instructions: some 26 for a lane's word of weights, 14 of them the widening and the product, at
// half an instruction a cycle. 8 tokens (42 experts): 71 us, 16 tokens: 101; in nvfp4 26, 80 and 107 to 115 (280 MB,
// 41 us), in mxfp4 24.5 for one and 102 for 16. (Measured beside it: a
// second CTA on an SM, with two groups or 64 registers a thread, 34 and 42 us where this took 26;
// a last unit cut among the groups, the same, as the instructions remain; the next piece's activations
// fetched behind this one's products, the same.)
//
// Every sum has a fixed order: outputs are the same every time.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "moe_chosen.cuh"
#include "tc.cuh"
#include "tiles.cuh"

namespace w4 {
namespace {

constexpr int kGroups = 4, kGroupWarps = 4, kGroupThreads = 128, kThreads = kGroups * kGroupThreads;
constexpr int kChunkSteps = 16;                      // steps of 32 columns in a ring slot
constexpr int kPer = kChunkSteps / kGroupWarps;      // a warp's of them
constexpr int64_t kMaxI = 1 << 20;                   // 256 experts of I / 16 units times 152 CTAs are numbers of 32 bits
constexpr int kRows = 32;                            // weight rows of a unit
constexpr int kBox = kRows * 128;                    // 8 steps of them, 128-byte swizzle: 16-byte chunk c of row r at c ^ r % 8
constexpr int kSlot = kChunkSteps / 8 * kBox;

struct Params {
  CUtensorMap tm_w;        // up: [2E, I, K/2 bytes] in boxes of 16 rows of two matrices; down: [E, H, K/2 bytes], 32 rows
  CUtensorMap tm_s;        // by_piece: the scales alike, scale_pitch bytes a row
  MoeRouteArgs route;      // ids and wts unset
  const uint8_t* w_scale;  // [E, rows, scale_row bytes]
  const float* w_global;   // [E] or null
  const uint16_t* x;       // up: bf16 [T, H]
  uint4* choice;           // the up kernel's, for the down kernel
  uint16_t* act;           // fp16 [pairs, 2, I]
  uint8_t* act_exp;        // [pairs, I / 8]: biased exponents
  uint16_t* y;             // down: bf16 [T, H]
  int H, I, K, rows;       // K: columns of w (up: H, down: I); rows an expert
  int group_steps, group_shift;   // int4: 32-column steps of a scale; their logarithm, or -1
  bool by_piece;           // scales come by the piece, else whole rows of them by the unit
  int scale_row;           // bytes of a row's scales
  int scale_pitch;         // of a row's in shared memory
  int chunks, slots, scale_slots;
  int split;               // down: CTAs of a cluster that share the experts of a slice
  unsigned int* status;
};

// fp16 pairs of the 8 weights of a word; sc: the block's scale twice (nvfp4).
// int4: columns (0,4), (1,5), (2,6), (3,7); else (0,1), (2,3), (4,5), (6,7).
template <int kFmt>
W4_DEV void widen(uint32_t w, uint32_t sc, uint32_t (&d)[4]) {
  if constexpr (kFmt == W4_FMT_INT4) {
    constexpr uint32_t k1024 = 0x64006400u, k1032 = 0x64086408u, kSixteenth = 0x2C002C00u, kMinus72 = 0xD480D480u;
    const uint32_t v = w >> 8;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d[0]) : "r"(and_or(w, 0x000F000Fu, k1024)), "r"(k1032));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d[1]) : "r"(and_or(w, 0x00F000F0u, k1024)), "r"(kSixteenth), "r"(kMinus72));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d[2]) : "r"(and_or(v, 0x000F000Fu, k1024)), "r"(k1032));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d[3]) : "r"(and_or(v, 0x00F000F0u, k1024)), "r"(kSixteenth), "r"(kMinus72));
  } else {
    e2m1x8_to_f16(w, d);
    if constexpr (kFmt == W4_FMT_NVFP4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(d[i]) : "r"(sc));
    }
  }
}

// Place of column i (of 8) in an activation's chunk, to match widen.
template <int kFmt>
W4_DEV int chunk_place(int i) {
  return kFmt == W4_FMT_INT4 ? (i & 3) * 2 + (i >> 2) : i;
}

W4_DEV void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same on zeros.
W4_DEV void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

W4_DEV void group_sync(int group) { asm volatile("bar.sync %0, %1;" :: "r"(group + 1), "r"(kGroupThreads) : "memory"); }

// x_t as fp16 times a power of two, by one warp; returns what undoes it.
template <int kFmt>
W4_DEV float widen_row(const Params& p, int t, uint8_t* to) {
  const int lane = threadIdx.x & 31;
  const uint4* xr = reinterpret_cast<const uint4*>(p.x) + static_cast<size_t>(t) * (p.H / 8);
  const int n = p.H / 8;
  // eight chunks a lane at a time, that their loads are in flight together; those of 2048 columns stay for the second pass
  constexpr int kAtOnce = 8;
  uint4 v[kAtOnce];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + 32 * k + lane;
      v[k] = i < n ? ld_cg_v4(xr + i) : make_uint4(0, 0, 0, 0);
    }
  };
  uint32_t m = 0;
  int i0 = 0;
#pragma unroll 1
  for (;; i0 += 32 * kAtOnce) {
    fetch(i0);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      m = __vmaxu2(__vmaxu2(m, v[k].x & 0x7FFF7FFFu), v[k].y & 0x7FFF7FFFu);
      m = __vmaxu2(__vmaxu2(m, v[k].z & 0x7FFF7FFFu), v[k].w & 0x7FFF7FFFu);
    }
    if (i0 + 32 * kAtOnce >= n) break;
  }
  m = __reduce_max_sync(kFull, max(m & 0xFFFFu, m >> 16));
  const int e = max(static_cast<int>(m >> 7), 15);   // biased exponent; factors are normal numbers
  const float f = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);   // 2^(14 - (e - 127))
#pragma unroll 1
  for (;; i0 -= 32 * kAtOnce) {   // the last ones are here
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + 32 * k + lane;
      float a[8];
      chunk_f32<false>(v[k], a);
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int lo = kFmt == W4_FMT_INT4 ? j : 2 * j, hi = kFmt == W4_FMT_INT4 ? j + 4 : 2 * j + 1;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[j]) : "f"(a[hi] * f), "f"(a[lo] * f));
      }
      if (i < n) *reinterpret_cast<uint4*>(to + i * 16) = make_uint4(h[0], h[1], h[2], h[3]);
    }
    if (i0 == 0) break;
    fetch(i0 - 32 * kAtOnce);
  }
  return __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
}

// Where a group is in its list of units: chosen expert and first row. A unit is two blocks
// of 16 rows, one behind the other (down) or gate and up.
template <bool kDown>
struct Place {
  int a, n0, left;   // left: units from here to the end of the CTA's list, before which it stands while positive
  W4_DEV void skip(int I, int units) {
    left -= units;
    if constexpr (kDown) {
      a += units;
    } else {
      n0 += 16 * units;
      while (n0 >= I) n0 -= I, ++a;
    }
  }
};

// 2^e, -127 <= e <= 127: the least is not a normal number.
W4_DEV float two_to(int e) { return __uint_as_float(e == -127 ? 0x00400000u : static_cast<uint32_t>(e + 127) << 23); }
W4_DEV uint32_t e4m3_f16x2(uint32_t s8) { return e4m3x2_to_f16x2(s8 * 0x0101u); }   // twice
// Powers of two of two bytes, in the low ones first: 2^(byte - 127), NaN for 255.
W4_DEV uint32_t e8m0x2_bf16x2(uint32_t two) {
  uint32_t d;
  asm("{.reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.bf16x2.ue8m0x2 %0, t;}" : "=r"(d) : "r"(two));
  return d;
}
W4_DEV float scale_int4(const uint8_t* row, int grp) { return half_bits_to_f32(reinterpret_cast<const uint16_t*>(row)[grp]); }

// Where this lane's two MMA blocks find their rows: block m has rows r, r + 8 of the MMA from
// rows at[m], at[m] + apart of the unit.
template <bool kDown>
struct RowsOf {
  static constexpr int kApart = kDown ? 8 : 16;
  W4_DEV static int first(int m) { return kDown ? 16 * m : 8 * m; }
};

// Adds this warp's steps [s0, s1), at most kPer, to y[block]; the slot starts at step c0, the scales at step z0. b(i)
// are the lane's 8 activations of step s0 + i (columns 8 (lane % 4) ..) of column lane / 4 of the block.
// kWhole: int4, kPer steps that have one scale.
template <int kFmt, bool kDown, bool kWhole, class B>
W4_DEV void multiply(const Params& p, const uint8_t* slot, const uint8_t* scales, int c0, int z0, int s0, int s1, B b,
                     float (&y)[2][4]) {
  using R = RowsOf<kDown>;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const uint8_t* w0 = slot + g * 128 + 4 * c;
  const uint32_t swz = static_cast<uint32_t>(g) << 4;
  const uint8_t* sc[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) sc[m][h] = scales + (R::first(m) + h * R::kApart + g) * p.scale_pitch;
  // one step: weights to operand registers, two products a block; with `zero`, d is written
  auto step = [&](int s, const uint4& v, const uint32_t (&f)[2][2], float (&d)[2][4], bool zero) {
    const uint8_t* w = w0 + ((s - c0) >> 3) * kBox + (((static_cast<uint32_t>(s) & 7u) << 4) ^ swz);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint32_t ra[4], rb[4];
      widen<kFmt>(*reinterpret_cast<const uint32_t*>(w + R::first(m) * 128), f[m][0], ra);
      widen<kFmt>(*reinterpret_cast<const uint32_t*>(w + (R::first(m) + R::kApart) * 128), f[m][1], rb);
      if (zero)
        mma16816_zero(d[m], ra[0], rb[0], ra[1], rb[1], v.x, v.y);
      else
        mma16816(d[m], ra[0], rb[0], ra[1], rb[1], v.x, v.y);
      mma16816(d[m], ra[2], rb[2], ra[3], rb[3], v.z, v.w);
    }
  };
  auto add = [&](const float (&f)[2][2], const float (&d)[2][4]) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      y[m][0] = fmaf(f[m][0], d[m][0], y[m][0]), y[m][1] = fmaf(f[m][0], d[m][1], y[m][1]);
      y[m][2] = fmaf(f[m][1], d[m][2], y[m][2]), y[m][3] = fmaf(f[m][1], d[m][3], y[m][3]);
    }
  };
  if constexpr (kFmt == W4_FMT_NVFP4) {
    if (s1 - s0 == kPer && (s0 & 1) == 0) {   // scales of two steps are a word (a row's are multiples of 4 bytes)
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        uint32_t word[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) word[m][h] = reinterpret_cast<const uint32_t*>(sc[m][h])[(s0 - z0 + i) >> 1];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t f[2][2];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) f[m][h] = e4m3x2_to_f16x2(prmt(word[m][h], 0, (c >> 1) * 0x11 + j * 0x22 + 0x4400));
          step(s0 + i + j, b(i + j), f, y, false);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (s0 + i >= s1) break;
        uint32_t f[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) f[m][h] = e4m3_f16x2(sc[m][h][2 * (s0 - z0 + i) + (c >> 1)]);
        step(s0 + i, b(i), f, y, false);
      }
    }
  } else if constexpr (kFmt == W4_FMT_MXFP4) {
    const uint32_t none[2][2] = {};
    if (s1 - s0 == kPer && (p.scale_pitch & 3) == 0) {   // scales of four steps are a word
      static_assert(kPer == 4, "a word of scales");
      uint32_t word[2][2];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) word[m][h] = *reinterpret_cast<const uint32_t*>(sc[m][h] + s0 - z0);
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        float d[2][4], f[2][2][2];   // f: [step]
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t two = e8m0x2_bf16x2(word[m][h] >> (8 * i));
            f[0][m][h] = bf16_lo(two), f[1][m][h] = bf16_hi(two);
          }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          step(s0 + i + j, b(i + j), none, d, true);
          add(f[j], d);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (s0 + i >= s1) break;
        float d[2][4], f[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) f[m][h] = bf16_lo(e8m0x2_bf16x2(sc[m][h][s0 - z0 + i]));
        step(s0 + i, b(i), none, d, true);
        add(f, d);
      }
    }
  } else {
    const uint32_t none[2][2] = {};
    float d[2][4], f[2][2];
    auto scales_of = [&](int grp) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) f[m][h] = scale_int4(sc[m][h], grp);
    };
    int grp = kWhole || p.group_shift >= 0 ? (s0 - z0) >> p.group_shift : (s0 - z0) / p.group_steps;
    scales_of(grp);
    const int end = z0 + (grp + 1) * p.group_steps;
    if (kWhole || (s1 - s0 == kPer && s1 <= end)) {   // one scale for all
#pragma unroll
      for (int i = 0; i < kPer; ++i) step(s0 + i, b(i), none, d, i == 0);
      add(f, d);
      return;
    }
    int left = end - s0;
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j >> 2][j & 3] = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (s0 + i >= s1) break;
      step(s0 + i, b(i), none, d, false);
      if (--left == 0 || s0 + i + 1 == s1) {   // the end of a scale's columns, or of this warp's
        add(f, d);
        if (s0 + i + 1 == s1) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j >> 2][j & 3] = 0.f;
        scales_of(++grp);
        left = p.group_steps;
      }
    }
  }
}

// Shared memory beyond Routed: barriers, sums of the groups' warps, then (dynamic) the rings
// of row pieces and of scales, and up: x in fp16, down: each group's outputs.
struct Common {
  Routed r;
  alignas(16) float red[kGroups][2][kGroupWarps][2][32][4];   // [group][in turn][warp][block][lane]
  uint64_t full[kGroups][kMoeDecodeSlots];
  uint64_t empty[kGroups][kMoeDecodeSlots];   // a group's warps are done with a slot
  int abort_flag;
};

// In front of the shared memory.
W4_DEV Common& common_of(uint8_t* smem_dyn) {
  return *reinterpret_cast<Common*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
}
// By all threads, before the wait for the kernels before.
W4_DEV void prepare(const Params& p, Common& c) {
  if (threadIdx.x == 0) {
    for (int g = 0; g < kGroups; ++g)
      for (int i = 0; i < p.slots; ++i) {
        mbar_init(&c.full[g][i], 1);
        mbar_init(&c.empty[g][i], kGroupWarps);
      }
    c.abort_flag = 0;
    fence_mbar_init();
  }
}

// A kernel behind that wait. kBlocks: of an expert's tokens, 8 of them (up) or 4 (down, whose
// activations are pairs of columns). kWhole: as multiply.
template <int kFmt, bool kDown, int kBlocks, bool kWhole>
W4_DEV void layer(const Params& p, Common& c) {
  uint8_t* smem = reinterpret_cast<uint8_t*>(&c);
  constexpr int kTokens = kDown ? 4 : 8, kSums = kDown ? 2 : 4;   // of a block, a lane's sums of 16 rows
  Routed& r = c.r;
  uint8_t* ring = smem + (sizeof(Common) + 1023) / 1024 * 1024;
  uint8_t* scale_ring = ring + kGroups * p.slots * kSlot;
  const int scale_slot = kRows * p.scale_pitch;
  uint8_t* rest = scale_ring + kGroups * p.scale_slots * scale_slot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = static_cast<int>(p.route.T);
  volatile int* abort_flag = &c.abort_flag;

  const int x_pitch = 2 * p.H + 64;   // two tokens' pieces lie in different banks
  if constexpr (kDown) {
    take_choice<kThreads>(r, p.choice);
  } else {
    route_prepare<kThreads>(r);
    route_all<kThreads>(p.route, r, reinterpret_cast<uint32_t*>(ring), [&](int w) {
      const int t = T <= 8 ? w - 8 : w;   // by warps that route no token, where there are
      if (t >= 0 && t < T) {
        const float f = widen_row<kFmt>(p, t, rest + t * x_pitch);
        if (lane == 0) r.x_scale[t] = f;
      }
    });
    if (blockIdx.x == 0) keep_choice<kThreads>(r, p.choice);
  }

  // units of this CTA: up, a share of all (expert, 16 columns) in order; down, every split-th expert.
  // A group takes every kGroups-th of them.
  const int rank = kDown && p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int stride = kGroups * (kDown ? p.split : 1), steps = p.K / 32;

  {
    const int group = warp / kGroupWarps, w = warp % kGroupWarps, tid = threadIdx.x % kGroupThreads;
    const int g = lane >> 2, q = lane & 3;
    const uint64_t policy = tc::evict_first_policy();   // weights are read once
    Place<kDown> at;
    if constexpr (kDown) {
      at.a = rank + group * p.split, at.n0 = static_cast<int>(blockIdx.x) / p.split * kRows, at.left = r.n - at.a;
    } else {
      const unsigned per = p.I / 16, all = r.n * per;   // times a CTA's index below 2^32: kMaxI
      const unsigned u0 = all * blockIdx.x / gridDim.x + group, u1 = all * (blockIdx.x + 1) / gridDim.x;
      at.a = u0 / per, at.n0 = (u0 - at.a * per) * 16, at.left = static_cast<int>(u1) - static_cast<int>(u0);
    }
    uint8_t* const my_ring = ring + group * p.slots * kSlot;
    uint8_t* const my_scales = scale_ring + group * p.scale_slots * scale_slot;
    // The next piece to copy. All warps of the group keep count.
    Place<kDown> to = at;
    int to_ch = 0, to_slot = 0, to_scale = 0;
    // A whole warp: starts the copies of that piece, with its scales, or its unit's scales with the first of the unit.
    auto fill = [&]() {
      if (to.left > 0 && elect_one()) {
        const int s0 = to_ch * kChunkSteps, boxes = (min(kChunkSteps, steps - s0) + 7) / 8, e = r.expert[to.a];
        uint64_t* bar = &c.full[group][to_slot];
        uint8_t* slot = my_ring + to_slot * kSlot;
        mbar_arrive_expect_tx(bar, boxes * kBox + (p.by_piece || to_ch == 0 ? scale_slot : 0));
        for (int i = 0; i < boxes; ++i)
          tc::tma_load_3d_hint(slot + i * kBox, &p.tm_w, bar, (s0 + 8 * i) * 16, to.n0, kDown ? e : 2 * e, policy);
        if (p.by_piece) {
          tc::tma_load_3d(my_scales + to_slot * scale_slot, &p.tm_s, bar, to_ch * p.scale_pitch, to.n0, kDown ? e : 2 * e);
        } else if (to_ch == 0) {
          uint8_t* sc = my_scales + to_scale * scale_slot;
          const uint8_t* from = p.w_scale + (static_cast<size_t>(e) * p.rows + to.n0) * p.scale_row;
          tc::bulk_load(sc, from, 16 * p.scale_row, bar);
          tc::bulk_load(sc + 16 * p.scale_row, from + static_cast<size_t>(kDown ? 16 : p.I) * p.scale_row, 16 * p.scale_row, bar);
        }
      }
      __syncwarp();
    };
    auto filled = [&]() {   // on to the piece after it
      if (++to_slot == p.slots) to_slot = 0;
      if (++to_ch == p.chunks) {
        to_ch = 0;
        if (++to_scale == p.scale_slots) to_scale = 0;
        to.skip(p.I, stride);
      }
    };
    tc::fence_proxy_async_smem();   // the ring held the routing's scratch
    for (int i = 0; i < p.slots; ++i) {
      if (w == (i & (kGroupWarps - 1))) fill();
      filled();
    }
    float* out = reinterpret_cast<float*>(rest) + group * T * kRows;   // down: [T][32]
    if constexpr (kDown) {
      for (int i = tid; i < T * kRows; i += kGroupThreads) out[i] = 0.f;
    }
    int count = 0, slot = 0, phase = 0, scale_at = 0, turn = 0;
    bool ok = true;
    for (; at.left > 0; at.skip(p.I, stride)) {
      const int first = r.first[at.a], tokens = r.first[at.a + 1] - first;
      const float gl = p.w_global != nullptr ? __ldcg(p.w_global + r.expert[at.a]) : 1.f;
      float y[kDown ? 1 : kBlocks][2][kSums] = {};   // [block of tokens][16 rows]
      // down: of the blocks behind the first, which few experts have (in local memory)
      float more[kDown && kBlocks > 1 ? kBlocks - 1 : 1][2][kSums];
      if constexpr (kDown && kBlocks > 1) {
        if (tokens > kTokens) {
#pragma unroll
          for (int i = 0; i < (kBlocks - 1) * 2 * kSums; ++i) more[i / (2 * kSums)][i / kSums % 2][i % kSums] = 0.f;
        }
      }
      for (int ch = 0; ch < p.chunks; ++ch, ++count) {
        const int c0 = ch * kChunkSteps;
        const int s0 = min(c0 + kPer * w, steps), s1 = min(s0 + kPer, steps);
        const uint8_t* piece = my_ring + slot * kSlot;
        const uint8_t* scales = my_scales + (p.by_piece ? slot : scale_at) * scale_slot;
        const int z0 = p.by_piece ? c0 : 0;
        // this lane's column of a block: a token, or half of its activations; columns past the last token repeat it
        auto row_of = [&](int nb) { return first + min(kTokens * nb + (kDown ? g >> 1 : g), tokens - 1); };
        uint4 v[kPer];
        int e[kPer];
        auto fetch = [&](int nb) {   // activations and their exponents
          const uint16_t* ar = p.act + (2 * static_cast<size_t>(row_of(nb)) + (g & 1)) * p.K + 8 * q;
          const uint8_t* er = p.act_exp + static_cast<size_t>(row_of(nb)) * (p.K / 8) + q;
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (kWhole ? s0 < s1 : s0 + i < s1) {
              v[i] = ld_cg_v4(ar + 32 * (s0 + i));
              e[i] = __ldcg(er + 4 * (s0 + i));
            }
        };
        if constexpr (kDown) fetch(0);
        // after a time-out the group goes on without waiting, so that its warps still meet
        ok = ok && wait_warp(&c.full[group][slot], phase, abort_flag, p.status);
        auto held = [](float& v) { asm volatile("" : "+f"(v) :: "memory"); };
        // one block of tokens: fold(m, h, v, f) takes this lane's sums
        auto block = [&](int nb, auto fold) {
          int top = 0, low = 255;
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (kWhole || s0 + i < s1) top = max(top, e[i]), low = min(low, e[i]);
          top = max(top, __shfl_xor_sync(kFull, top, 1));
          top = max(top, __shfl_xor_sync(kFull, top, 2));
          auto shift = [&](uint4& a, int by) {   // times 2^by, from 2^-24 on
            const float f = __uint_as_float(static_cast<uint32_t>(max(127 + by, 0)) << 23);
            uint32_t h;
            asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(h) : "f"(f));
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(a.x) : "r"(h));
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(a.y) : "r"(h));
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(a.z) : "r"(h));
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(a.w) : "r"(h));
          };
          if (__any_sync(kFull, top - low > 24)) {   // far apart: in two steps
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              if ((kWhole || s0 + i < s1) && top - e[i] > 24) {
                shift(v[i], -24);
                e[i] += 24;
              }
          }
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (kWhole || s0 + i < s1) shift(v[i], e[i] - top);
          float d[2][4] = {};
          multiply<kFmt, kDown, kWhole>(p, piece, scales, c0, z0, s0, s1, [&](int i) { return v[i]; }, d);
          // the lane's two columns are a token's halves: a factor 2^(top - 127 - 14), and 2^-11 of the second
          const float f = two_to(__shfl_sync(kFull, top, 8 * q) - 141);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float a = fmaf(d[m][2 * h + 1], 1.f / 2048.f, d[m][2 * h]);
              held(a);
              fold(m, h, a, f);
            }
        };
        if constexpr (kDown) {
          if (s0 < s1) {
            block(0, [&](int m, int h, float a, float f) { y[0][m][h] = fmaf(a, f, y[0][m][h]); });
            if constexpr (kBlocks > 1) {
#pragma unroll 1
              for (int nb = 1; kTokens * nb < tokens; ++nb) {
                fetch(nb);
                block(nb, [&](int m, int h, float a, float f) { more[nb - 1][m][h] = fmaf(a, f, more[nb - 1][m][h]); });
              }
            }
          }
        } else {
#pragma unroll
          for (int nb = 0; nb < kBlocks; ++nb) {
            if (kTokens * nb >= tokens || s0 >= s1) break;
            const uint8_t* xr = rest + r.token[row_of(nb)] * x_pitch + 64 * s0 + 16 * q;
            multiply<kFmt, kDown, kWhole>(p, piece, scales, c0, z0, s0, s1,
                                          [&](int i) { return *reinterpret_cast<const uint4*>(xr + 64 * i); }, y[nb]);
#pragma unroll
            for (int k = 0; k < 8; ++k) held(y[nb][k >> 2][k & 3]);
          }
        }
        // the slot goes back behind the products that used its words and the scales (taken in `held`), with
        // a fence between them and the next copy
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.empty[group][slot]);
        // One of the warps copies the next piece into the place of the one before this, which the
        // others left a piece ago or soon will.
        if (count > 0) {
          if (w == (count & (kGroupWarps - 1))) {
            const int last = slot == 0 ? p.slots - 1 : slot - 1;
            ok = ok && wait_warp(&c.empty[group][last], slot == 0 ? phase ^ 1 : phase, abort_flag, p.status);
            if (ok) fill();
          }
          filled();
        }
        if (++slot == p.slots) slot = 0, phase ^= 1;
      }
      if (++scale_at == p.scale_slots) scale_at = 0;
      // the warps' sums z of a block of tokens meet
      auto meet = [&](int nb, const float (&z)[2][kSums]) {
        float (*red)[2][32][4] = c.red[group][turn];   // two in turn, so that one meeting is enough
        turn ^= 1;
        if constexpr (kDown) {
          *reinterpret_cast<float4*>(red[w][0][lane]) = make_float4(z[0][0], z[0][1], z[1][0], z[1][1]);
        } else {
#pragma unroll
          for (int m = 0; m < 2; ++m) *reinterpret_cast<float4*>(red[w][m][lane]) = make_float4(z[m][0], z[m][1], z[m][2], z[m][3]);
        }
        group_sync(group);
        auto sum = [&](int m, int l, int j) { return ((red[0][m][l][j] + red[1][m][l][j]) + red[2][m][l][j]) + red[3][m][l][j]; };
        if constexpr (kDown) {
          // thread: column tid % 32 of the unit, token tid / 32, a warp's own
          const int o = lane, n = 4 * nb + w;
          if (n < tokens) {
            const float v = sum(0, (o & 7) * 4 + w, o >> 3);
            float& at = out[r.token[first + n] * kRows + o];
            at = fmaf(v, gl * r.weight[first + n], at);
          }
        } else if (8 * nb + 2 * w < tokens) {   // a warp with no token has nothing to do here
          // thread: column tid % 16 of the unit, token tid / 16
          const int i = tid & 15, n = 8 * nb + (tid >> 4);
          const int k = min(n, tokens - 1), l = (i & 7) * 4 + (k & 7) / 2, j = k & 1;
          const float f = r.x_scale[r.token[first + k]];
          const float gate = sum(i >> 3, l, j) * f * gl, up = sum(i >> 3, l, 2 + j) * f * gl;
          const float a = __fdiv_rn(gate, 1.f + expf(-gate)) * up;
          uint32_t bits = __float_as_uint(a) & 0x7FFFFFFFu;
          bits = max(bits, __shfl_xor_sync(kFull, bits, 1));
          bits = max(bits, __shfl_xor_sync(kFull, bits, 2));
          bits = max(bits, __shfl_xor_sync(kFull, bits, 4));
          const uint32_t ex = max(bits >> 23, 14u);   // a 2^(14 - (ex - 127)): the largest in [2^14, 2^15)
          if (n < tokens) {
            // in two halves of 11 bits, the second 2^11 times what the first left
            const float f16 = a * __uint_as_float((268u - ex) << 23);
            uint16_t hi, lo;
            asm("cvt.rn.f16.f32 %0, %1;" : "=h"(hi) : "f"(f16));
            const float left = f16 - half_bits_to_f32(hi);
            asm("cvt.rn.f16.f32 %0, %1;" : "=h"(lo) : "f"(left == left ? left * 2048.f : 0.f));   // of an infinity nothing
            uint16_t* to = p.act + 2 * static_cast<size_t>(first + n) * p.I + at.n0 + (i & 8) + chunk_place<kFmt>(i & 7);
            to[0] = hi, to[p.I] = lo;
            if ((i & 7) == 0) p.act_exp[static_cast<size_t>(first + n) * (p.I / 8) + (at.n0 + i) / 8] = static_cast<uint8_t>(ex);
          }
        }
      };
      if constexpr (kDown) {
        meet(0, y[0]);
        if constexpr (kBlocks > 1) {
#pragma unroll 1
          for (int nb = 1; kTokens * nb < tokens; ++nb) meet(nb, more[nb - 1]);
        }
      } else {
#pragma unroll
        for (int nb = 0; nb < kBlocks; ++nb) {
          if (kTokens * nb >= tokens) break;
          meet(nb, y[nb]);
        }
      }
    }
  }

  if constexpr (kDown) {
    __syncthreads();
    // the groups' outputs in order, then (split) the CTAs' of the cluster
    float* sum = reinterpret_cast<float*>(rest);
    for (int i = threadIdx.x; i < T * kRows; i += kThreads) {
      float v = sum[i];
      for (int g = 1; g < kGroups; ++g) v += sum[g * T * kRows + i];
      sum[i] = v;
    }
    if (p.split > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    const int n0 = static_cast<int>(blockIdx.x) / p.split * kRows;
    const int i = threadIdx.x * 4;
    if (rank == 0 && i < T * kRows) {
      float4 v = *reinterpret_cast<const float4*>(sum + i);
      for (int k = 1; k < p.split; ++k) {
        const float4 o = ld_cluster_f32x4(smem_addr(sum + i), k);
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
      }
      *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(i / kRows) * p.H + n0 + i % kRows) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
    if (p.split > 1) {
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    }
  }
  if (*abort_flag) {   // let copies in flight land before the shared memory goes away
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 1000000ull) {
    }
  }
}

// Bytes of a row's scales.
int scale_row_bytes(const MoeDecodeArgs& a, bool down) {
  const int64_t K = down ? a.I : a.H;
  return static_cast<int>(a.format == W4_FMT_INT4 ? 2 * (K / (down ? a.down_group : a.gate_up_group)) : a.format == W4_FMT_NVFP4 ? K / 16 : K / 32);
}

// Of a piece's columns, where TMA takes rows of scales in whole pieces; else 0.
int scale_piece_bytes(const MoeDecodeArgs& a, bool down) {
  constexpr int kColumns = 32 * kChunkSteps;
  const int group = a.format == W4_FMT_INT4 ? (down ? a.down_group : a.gate_up_group) : static_cast<int>(fp4_block(a.format == W4_FMT_NVFP4));
  const int bytes = kColumns % group == 0 ? kColumns / group * (a.format == W4_FMT_INT4 ? 2 : 1) : 0;
  return bytes % 16 == 0 && scale_row_bytes(a, down) % 16 == 0 ? bytes : 0;
}

// Shared memory: `slots` ring slots a group, the most that fit; fewer than two: it does not fit.
struct Layout {
  int slots, chunks, scale_slots, scale_pitch;
  bool by_piece;
  int64_t bytes;
};
Layout layout_of(const MoeDecodeArgs& a, bool down) {
  const int64_t K = down ? a.I : a.H, T = a.route.T;
  const int64_t rest = down ? kGroups * T * kRows * 4 : T * (2 * a.H + 64);
  Layout l;
  l.chunks = static_cast<int>((K / 32 + kChunkSteps - 1) / kChunkSteps);
  l.scale_pitch = scale_piece_bytes(a, down);
  l.by_piece = l.scale_pitch > 0;
  if (!l.by_piece) l.scale_pitch = scale_row_bytes(a, down);
  for (l.slots = kMoeDecodeSlots; l.slots >= 2; --l.slots) {
    l.scale_slots = l.by_piece ? l.slots : (l.slots + l.chunks - 1) / l.chunks + 1;   // a unit's are in use until its last piece is done
    l.bytes = 1024 + static_cast<int64_t>(sizeof(Common) + 1023) / 1024 * 1024 + rest +
              static_cast<int64_t>(kGroups) * (l.slots * kSlot + static_cast<int64_t>(l.scale_slots) * kRows * l.scale_pitch);
    if (l.bytes <= 232448) break;
  }
  return l;
}

// kKernel: of weights in kFmt.
template <auto kKernel, int kFmt, bool kDown>
cudaError_t run(const MoeDecodeArgs& a, cudaStream_t s) {
  const Layout l = layout_of(a, kDown);
  if (l.slots < 2) return cudaErrorInvalidConfiguration;   // refused before (moe_decode_fits)
  Params p = {};
  p.route = a.route;
  const int T = static_cast<int>(a.route.T);
  cudaError_t e = kDown ? encode(&p.tm_w, a.down, a.I / 2, a.H, a.route.E, kRows) : encode(&p.tm_w, a.gate_up, a.H / 2, a.I, 2 * a.route.E, kRows / 2, 2);
  if (e == cudaSuccess && l.by_piece)
    e = kDown ? encode(&p.tm_s, a.down_scale, scale_row_bytes(a, true), a.H, a.route.E, kRows, 1, l.scale_pitch)
              : encode(&p.tm_s, a.gate_up_scale, scale_row_bytes(a, false), a.I, 2 * a.route.E, kRows / 2, 2, l.scale_pitch);
  if (e != cudaSuccess) return e;
  p.w_scale = static_cast<const uint8_t*>(kDown ? a.down_scale : a.gate_up_scale);
  p.w_global = kDown ? a.down_global : a.gate_up_global;
  p.x = static_cast<const uint16_t*>(a.x);
  p.choice = static_cast<uint4*>(a.workspace);
  p.act = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.workspace) + kMoeChoiceBytes);
  p.act_exp = reinterpret_cast<uint8_t*>(p.act + 2 * static_cast<size_t>(T) * a.route.k * a.I);
  p.y = static_cast<uint16_t*>(a.y);
  p.H = static_cast<int>(a.H);
  p.I = static_cast<int>(a.I);
  p.K = kDown ? p.I : p.H;
  p.rows = kDown ? p.H : 2 * p.I;
  p.group_steps = kFmt == W4_FMT_INT4 ? (kDown ? a.down_group : a.gate_up_group) / 32 : 1;
  p.group_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (p.group_steps == 1 << i) p.group_shift = i;
  p.scale_row = scale_row_bytes(a, kDown);
  p.by_piece = l.by_piece, p.scale_pitch = l.scale_pitch;
  p.slots = l.slots, p.chunks = l.chunks, p.scale_slots = l.scale_slots;
  p.status = a.status;
  p.split = 1;
  int64_t grid = current_sm_count();
  if (kDown) {
    const int64_t slices = p.H / kRows;
    for (int n = kMaxSplit; n > 1 && p.split == 1; n /= 2)
      if (slices * n <= grid && n <= a.route.k * T) p.split = n;
    grid = slices * p.split;
  }
  return start<kKernel>(p, grid, kThreads, static_cast<int>(l.bytes), p.split, s, 232448);
}

}  // namespace
}  // namespace w4
