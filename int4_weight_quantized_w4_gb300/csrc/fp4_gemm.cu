// The microscaled 4-bit floating point product on the 5th-generation tensor cores
// (tcgen05, kind::mxf4 and kind::mxf4nvf4, sm_103a), dense and over expert segments
// of rows:
//
//   y[r, n] = bf16( g sum_b sx[r, b] sw[n, b] sum_{k in block b} q[r, k] w[n, k] + bias[n] ),
//
// q, w e2m1; blocks of 32 columns with power-of-two scales (mxfp4), or of 16 with e4m3
// scales and g the product of the two tensors' fp32 scales (nvfp4). The tensor core
// applies the block scales itself and sums in fp32, so that one accumulation runs over
// all of k and the epilogue is a multiply-add and one rounding.
//
// Operands come by TMA, 256 columns (128 bytes a row) a stage. Scales are row-major in
// memory, as checkpoints hold them; the MMA wants them in tensor memory, 128 rows' 32-bit
// words in four columns. They are copied 32 bytes a row at a time (two stages' nvfp4 scales,
// four stages' mxfp4), a warp per 128 rows transposes a stage's words in registers, and the
// MMA warp sends each 512-byte atom on to tensor memory ahead of the MMAs that use it.
//
// Two forms:
//  * stream (few rows): weights on the MMA's 128 rows, X tokens on its columns; dense
//    products share a tile's k among the CTAs of a cluster. Bound by the weight bytes.
//  * tile (many rows): 128 tokens on the MMA's rows, 192 outputs on its columns, with two
//    accumulators, so that the MMAs of a tile run while the one before leaves.
//    (Pairs of CTAs with cta_group::2 take in fewer bytes a stage, 33 KB for 45, but their arrivals on the
//    other CTA's barriers have to release at cluster scope: 204 us where tiles take 92.)
//
// All are launched as programmatic dependents and let their own dependents go early: the
// weights and their scales start while the kernels before finish, everything else waits.
#include <cstring>

#include "common.cuh"
#include "fp4_codes.cuh"
#include "fp4_scales.cuh"
#include "launch.h"
#include "tc.cuh"
#include "tiles.cuh"

namespace w4 {
namespace {

// Up to this many dense rows the stream form quantizes activations itself: one launch less.
constexpr int kFuseRows = 8;
constexpr int kQuantWarps = 4;                // that take the stages in turn

enum Form { kStream, kTile };

struct Params {
  CUtensorMap tm_x;        // codes [rows, K/2 bytes]
  CUtensorMap tm_w;        // codes [E, N, K/2 bytes]
  CUtensorMap tm_xs;       // scales [rows, SB], [E, N, SB], where tma_scales
  CUtensorMap tm_ws;
  const uint8_t* x_scale;
  const uint8_t* w_scale;
  const uint4* x;          // 16-bit activations [rows, K] to quantize, or null
  bool x_f16, x_wide;      // x_wide: 32-byte aligned
  const float* x_global;   // or null
  const float* w_global;   // [E], or null
  const uint16_t* bias;    // bf16 [N] or null
  uint16_t* y;             // bf16 [rows, N]
  const int32_t* offsets;  // [E + 1], or null (dense: one segment of all rows)
  int E, rows, N, K, SB, KS, n_tiles;   // SB: scale bytes a row, KS: stages over k
  bool tma_scales;         // rows of scales are 16-byte aligned; else words are copied one by one
  int split;               // stream form, dense: parts of the stages, one per CTA of a cluster
  int items;
  unsigned int* status;
};

// What a call's tiles follow from (tiles.cuh). offsets: a copy in shared memory where there
// is room, because every warp looks them up for every tile (from L2, 1300 cycles in which
// the MMAs of a 4096-token gate_up stood still).
struct Segments {
  const int32_t* offsets;
  int E, rows, n_tiles;
};
// Rows [a, b) of expert e; a segment outside [0, rows) counts as clipped.
W4_DEV void seg_bounds(const Segments& p, int e, int& a, int& b) {
  a = max(p.offsets[e], 0);
  b = min(p.offsets[e + 1], p.rows);
}

// W: weight rows of a tile, X: tokens of a CTA's tile.
template <int W, int X, bool kNv, Form kForm, bool kQuant = false>
struct Shape {
  static constexpr int WORDS = kNv ? 4 : 2;                    // 32-bit scale words of a row's stage
  static constexpr int SUPER = 8 / WORDS;                      // stages of a row's 32 bytes of scales
  static constexpr int N = kForm == kStream ? X : W;           // MMA columns
  static constexpr int AW = (W + 127) / 128, AX = (X + 127) / 128;   // atoms of 128 rows
  static constexpr int W_BYTES = W * kStageBytes, X_BYTES = X * kStageBytes;
  static constexpr int STAGE = W_BYTES + X_BYTES;
  static constexpr int SW_BYTES = AW * WORDS * 512, SSTAGE = SW_BYTES + AX * WORDS * 512;
  static constexpr int RAW_W = 128 * AW * 32, RAW = RAW_W + (X + 31) / 32 * 32 * 32;   // scales as they are in memory
  static constexpr int CTAS = kForm != kStream || X > 64 ? 1 : 2;   // resident per SM
  static constexpr int STAGES = CTAS == 2 ? (X == 64 ? 3 : 4) : kForm == kTile ? 4 : 5;
  static constexpr int RAWS = kForm != kStream || X == 32 ? 2 : 3;
  static constexpr int ACCS = 2;
  static constexpr int S_COLS = 4 * WORDS * (AW + AX);         // tensor memory columns of a stage's scales
  static constexpr int USED = ACCS * N + 2 * S_COLS;
  static constexpr int TMEM_COLS = USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
  static constexpr int EPI = 4;                                // epilogue warps: a quarter of the lanes each
  static constexpr int THREADS = 32 * (EPI + 4 + AW + AX + (kQuant ? kQuantWarps - 2 : 0));   // quantizers for a copying and a transposing warp
  static constexpr int OUT = kForm != kStream ? EPI * 2048 : 0;
  static constexpr int BARS = 2 * STAGES + 2 * RAWS + 2 * ACCS;
  static constexpr int STARTS = (kForm != kStream ? 2 : 1) * (kMaxExperts + 1) + 16;   // words
  static constexpr int SMEM = STAGES * (STAGE + SSTAGE) + RAWS * RAW + OUT + 256 + (STARTS + 3) / 4 * 16 + 1024;
  static_assert(USED <= 512 && CTAS * TMEM_COLS <= 512, "tensor memory");
  static_assert(SMEM <= 232448 && CTAS * SMEM + CTAS * 1024 <= 233472, "shared memory");
  static_assert(BARS * 8 + 8 <= 256, "barriers");
  static_assert(STAGE % 1024 == 0 && W_BYTES % 1024 == 0, "swizzle atoms");
  static_assert(kForm != kStream || X * 512 <= STAGES * STAGE, "part sums of a cluster fit the ring");
  // A quantizer sees every fourth phase of a stage's barrier; what it waited for before is at
  // most one phase back, so that a parity names one phase.
  static_assert(!kQuant || STAGES >= kQuantWarps, "see above");
};

template <int W, int X, bool kNv, Form kForm, bool kQuant = false>
__global__ void __launch_bounds__(Shape<W, X, kNv, kForm, kQuant>::THREADS, Shape<W, X, kNv, kForm, kQuant>::CTAS)
fp4_kernel(const __grid_constant__ Params p) {
  using C = Shape<W, X, kNv, kForm, kQuant>;
  // warps; below kMma: epilogue; kTurn ..: one per scale atom
  constexpr int kMma = C::EPI, kLoadW = kMma + 1, kLoadX = kQuant ? -1 : kMma + 2, kLoadS = kMma + 2 + !kQuant, kTurn = kLoadS + 1;
  constexpr int kQuant0 = kTurn + C::AW;   // kQuant: in the place of kLoadX and the activations' kTurn
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;                               // per stage: weights, activations
  uint8_t* scales = ring + C::STAGES * C::STAGE;      // per stage: weights', activations'
  uint8_t* raw = scales + C::STAGES * C::SSTAGE;      // per slot: weights', activations'
  uint4* out_base = reinterpret_cast<uint4*>(raw + C::RAWS * C::RAW);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(out_base) + C::OUT);
  uint64_t* empty = full + C::STAGES;
  uint64_t* raw_full = empty + C::STAGES;
  uint64_t* raw_empty = raw_full + C::RAWS;
  uint64_t* acc_full = raw_empty + C::RAWS;
  uint64_t* acc_empty = acc_full + C::ACCS;                                                   
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_empty + C::ACCS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int32_t* starts = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(full) + 256);
  int32_t* warp_sum = starts + kMaxExperts + 1;
  int32_t* offsets = warp_sum + 16;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], kQuant ? 2 + C::AW : 2 + C::AW + C::AX);   // operands; scale warps
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::RAWS; ++i) {
      mbar_init(&raw_full[i], p.tma_scales ? 1 : 32);
      mbar_init(&raw_empty[i], kQuant ? C::AW : C::AW + C::AX);
    }
    for (int i = 0; i < C::ACCS; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], C::EPI);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMma) tc::tmem_alloc(tmem_holder, C::TMEM_COLS);
  if (warp == kLoadW && lane == 0) tc::prefetch_tmap(&p.tm_w);
  if (warp == kLoadX && lane == 0) tc::prefetch_tmap(&p.tm_x);
  if (warp == kLoadS && lane == 0 && p.tma_scales) {
    tc::prefetch_tmap(&p.tm_ws);
    if (!kQuant) tc::prefetch_tmap(&p.tm_xs);
  }
  Segments seg{p.offsets, p.E, p.rows, p.n_tiles};
  if (p.offsets != nullptr) {
    grid_dependency_wait();   // the routing may be running still
    if constexpr (kForm != kStream) {
      for (int i = threadIdx.x; i <= p.E; i += C::THREADS) offsets[i] = p.offsets[i];
      seg.offsets = offsets;
      __syncthreads();
    }
    tile_starts<C::THREADS>(seg, X, starts, warp_sum);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  launch_dependents();
  const uint32_t tmem = *tmem_holder;

  // this CTA's part of the stages (the same for every item)
  const int part = p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int ks0 = p.KS * part / p.split, ks1 = p.KS * (part + 1) / p.split;
  const int first = blockIdx.x / p.split, step = gridDim.x / p.split;
  const int items = p.offsets == nullptr ? p.items : min(p.items, starts[p.E] * p.n_tiles);

  if (warp == kLoadW || warp == kLoadX) {
    // An operand.
    const bool is_w = warp == kLoadW;
    int st = 0, ph = 1, e = 0;
    bool ok = true, waited = !is_w;
    Tile t;
    if (!is_w) grid_dependency_wait();   // the codes come from the kernel before
    for (int it = first; ok && it < items && decode(seg, it, X, W, starts, t, e); it += step)
      for (int ks = ks0; ks < ks1; ++ks) {
        if (!waited && ph == 0) {   // the ring is full, and is emptied only after the kernels before
          grid_dependency_wait();
          waited = true;
        }
        if (!(ok = wait_warp(&empty[st], ph, abort_flag, p.status))) break;
        if (elect_one()) {
          uint8_t* to = ring + st * C::STAGE + (is_w ? 0 : C::W_BYTES);
          mbar_arrive_expect_tx(&full[st], is_w ? C::W_BYTES : C::X_BYTES);
          if (is_w)
            tc::tma_load_3d(to, &p.tm_w, &full[st], ks * kStageBytes, t.n0, t.expert);
          else
            tc::tma_load_2d(to, &p.tm_x, &full[st], ks * kStageBytes, t.row0);
        }
        __syncwarp();
        if (++st == C::STAGES) st = 0, ph ^= 1;
      }
  } else if (warp == kLoadS) {
    // Both operands' scales, 32 bytes a row; those that TMA cannot copy by all lanes.
    int rs = 0, rph = 1, e = 0;
    bool ok = true, waited = false;
    Tile t;
    for (int it = first; ok && it < items && decode(seg, it, X, W, starts, t, e); it += step) {
      for (int ks = ks0; ks < ks1; ks = (ks / C::SUPER + 1) * C::SUPER) {
        if (!(ok = wait_warp(&raw_empty[rs], rph, abort_flag, p.status))) break;
        uint8_t* to = raw + rs * C::RAW;
        const int at = ks / C::SUPER * 32;
        if (p.tma_scales) {
          if (elect_one()) {
            mbar_arrive_expect_tx(&raw_full[rs], 32 * (kQuant ? W : W + X));
            tc::tma_load_3d(to, &p.tm_ws, &raw_full[rs], at, t.n0, t.expert);
          }
          __syncwarp();
        } else {
          copy_scale_words(smem_addr(to), p.w_scale + (static_cast<size_t>(t.expert) * p.N + t.n0) * p.SB, p.SB, at, W, p.N - t.n0);
        }
        if (!waited) grid_dependency_wait();   // the activations' come from the kernel before
        waited = true;
        if (p.tma_scales) {
          if (!kQuant && elect_one()) tc::tma_load_2d(to + C::RAW_W, &p.tm_xs, &raw_full[rs], at, t.row0);
          __syncwarp();
        } else {
          if (!kQuant) copy_scale_words(smem_addr(to + C::RAW_W), p.x_scale + static_cast<size_t>(t.row0) * p.SB, p.SB, at, X, t.row_end - t.row0);
          tc::copy_async_arrive(&raw_full[rs]);
        }
        if (++rs == C::RAWS) rs = 0, rph ^= 1;
      }
    }
  } else if (kQuant && warp >= kQuant0) {
    // Quantizer w takes stages w, w + 4, ... of this CTA's sequence: lane l 16 columns, l % 16,
    // of rows l / 16 + 2 u. The next stage's columns are loaded as soon as this one's are used.
    if constexpr (kQuant) {
      const int h = lane >> 4, i = lane & 15, nks = ks1 - ks0;
      const int total = first < items ? (items - first + step - 1) / step * nks : 0;
      uint4 x[kFuseRows / 2][2];
      auto load = [&](int g) {
        const int c = (ks0 + g % nks) * 16 + i;   // in 16 columns
#pragma unroll
        for (int u = 0; u < kFuseRows / 2; ++u) {
          const int r = h + 2 * u;
          if (r < p.rows && 16 * c < p.K && g < total)
            load32(p.x + static_cast<size_t>(r) * (p.K / 8) + 2 * c, p.x_wide, x[u]);
          else
            x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
        }
      };
      grid_dependency_wait();   // x comes from the kernel before
      const float gx = kNv && p.x_global != nullptr ? *p.x_global : 1.f;
      load(warp - kQuant0);
      for (int g = warp - kQuant0; g < total; g += kQuantWarps) {
        const int st = g % C::STAGES;
        if (!wait_warp(&empty[st], ((g / C::STAGES) & 1) ^ 1, abort_flag, p.status)) break;
        uint8_t* to = ring + st * C::STAGE + C::W_BYTES + (i & 1) * 8;
        uint8_t* sc = scales + st * C::SSTAGE + C::SW_BYTES;
#pragma unroll
        for (int u = 0; u < kFuseRows / 2; ++u) {
          if (2 * u >= p.rows) break;
          const int r = h + 2 * u;   // a row past the last one fills a column that is never stored
          float f[2][8];
          uint32_t bits = p.x_f16 ? widen16<true>(x[u], f) : widen16<false>(x[u], f);
          if constexpr (!kNv) bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 1));
          uint2 code;
          const uint32_t s = block_codes<kNv>(f, bits, gx, code);
          *reinterpret_cast<uint2*>(to + r * 128 + (((i >> 1) ^ r) << 4)) = code;
          const int b = kNv ? i : i >> 1;   // byte of the stage's scales
          if (kNv || (i & 1) == 0) sc[(b >> 2) * 512 + r * 16 + (b & 3)] = static_cast<uint8_t>(s);
        }
        load(g + kQuantWarps);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
      }
    }
  } else if (warp >= kTurn) {
    // Lane l holds the words of rows l, l + 32, l + 64 and l + 96 of this warp's 128.
    const int a = warp - kTurn;
    const bool is_w = kQuant || a < C::AW;
    constexpr int kBlocksX = X < 128 ? (X + 31) / 32 : 4;
    const int blocks = is_w ? 4 : kBlocksX;
    const uint8_t* from = raw + (is_w ? a * 4096 : C::RAW_W + (a - C::AW) * 4096) + lane * 32;
    uint8_t* to = scales + (is_w ? a * 512 : C::SW_BYTES + (a - C::AW) * 512) + lane * 16;
    const int pitch = (is_w ? C::AW : C::AX) * 512;   // from word to word
    int st = 0, ph = 1, rs = 0, rph = 0, e = 0;
    bool ok = true;
    grid_dependency_wait();   // what it waits for depends on the kernels before
    Tile t;
    for (int it = first; ok && it < items && decode(seg, it, X, W, starts, t, e); it += step)
      for (int ks = ks0; ks < ks1; ++ks) {
        const int sub = ks % C::SUPER;
        if (ks == ks0 || sub == 0) {
          if (!(ok = wait_warp(&raw_full[rs], rph, abort_flag, p.status))) break;
        }
        uint32_t v[4][C::WORDS];
        load_scale_words<kNv>(from + rs * C::RAW + sub * C::WORDS * 4, blocks, v);
        if (!(ok = wait_warp(&empty[st], ph, abort_flag, p.status))) break;
        store_scale_atoms<kNv>(to + st * C::SSTAGE, pitch, v);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        // the slot goes back once its words have arrived in registers and the fence lies between them and the next copy
        if (ks == ks1 - 1 || sub == C::SUPER - 1) {
          if (lane == 0) mbar_arrive(&raw_empty[rs]);
          if (++rs == C::RAWS) rs = 0, rph ^= 1;
        }
        if (++st == C::STAGES) st = 0, ph ^= 1;
      }
  } else if (warp == kMma) {
    grid_dependency_wait();
    constexpr uint32_t idesc = tc::idesc_fp4<kNv>(128, C::N);
    const uint64_t wd0 = tc::sdesc_sw128(smem_addr(ring)), xd0 = wd0 + (C::W_BYTES >> 4);
    const uint64_t sd0 = tc::sdesc_scales(smem_addr(scales));
    int st = 0, ph = 0, ac = 0, aph = 1, buf = 0;
    bool ok = true;
    for (int it = first; ok && it < items; it += step) {
      if (!(ok = wait_warp(&acc_empty[ac], aph, abort_flag, p.status))) break;
      for (int ks = ks0; ks < ks1; ++ks) {
        if (!(ok = wait_warp(&full[st], ph, abort_flag, p.status))) break;
        tc::fence_after_sync();
        if (elect_one()) {
          // weights' scales, then the activations': [word][atom][4 columns] each
          const uint32_t sw = tmem + C::ACCS * C::N + buf * C::S_COLS, sx = sw + 4 * C::WORDS * C::AW;
          const uint64_t sd = sd0 + static_cast<uint64_t>((st * C::SSTAGE) >> 4);
#pragma unroll
          for (int i = 0; i < C::WORDS * (C::AW + C::AX); ++i) tc::copy_scales(sw + 4 * i, sd + 32 * i);
          const uint64_t wd = wd0 + static_cast<uint64_t>((st * C::STAGE) >> 4);
          const uint64_t xd = xd0 + static_cast<uint64_t>((st * C::STAGE) >> 4);
          const int left = p.K - ks * kStageK;
#pragma unroll
          for (int j = 0; j < 4; ++j) {   // 64 columns, 32 bytes, at a time
            if (64 * j >= left) break;
            const int word = kNv ? j : j >> 1;
            const uint32_t id = idesc | (kNv || !(j & 1) ? 0u : (2u << 29) | (2u << 4));
            const uint32_t fw = sw + 4 * C::AW * word, fx = sx + 4 * C::AX * word;
            const uint32_t acc = ks > ks0 || j > 0 ? 1u : 0u;
            if constexpr (kForm != kStream)
              tc::mma_fp4<kNv>(tmem + ac * C::N, xd + 2 * j, wd + 2 * j, id, fx, fw, acc);
            else
              tc::mma_fp4<kNv>(tmem + ac * C::N, wd + 2 * j, xd + 2 * j, id, fw, fx, acc);
          }
          tc::commit(&empty[st]);
          if (ks == ks1 - 1) tc::commit(&acc_full[ac]);
        }
        __syncwarp();
        buf ^= 1;
        if (++st == C::STAGES) st = 0, ph ^= 1;
      }
      if (++ac == C::ACCS) ac = 0, aph ^= 1;
    }
    __syncwarp();
  } else {
    grid_dependency_wait();   // the kernels before may still use y
    const float gx = p.x_global != nullptr ? __ldcg(p.x_global) : 1.f;
    int ac = 0, aph = 0, e = 0;
    bool ok = true;
    Tile t;
    auto hand_back = [&](int acc) {   // the accumulator is read
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
    };
    for (int it = first; ok && it < items && decode(seg, it, X, W, starts, t, e); it += step) {
      const float alpha = p.w_global != nullptr ? gx * __ldcg(p.w_global + t.expert) : gx;
      if (!(ok = wait_warp(&acc_full[ac], aph, abort_flag, p.status))) break;
      tc::fence_after_sync();
      const int q = warp & 3;
      const uint32_t ta = tmem + (static_cast<uint32_t>(32 * q) << 16) + ac * C::N;
      if constexpr (kForm != kStream) {
        const int row0 = t.row0 + 32 * q;
        uint4* buf = out_base + warp * 128;
        uint16_t* yp = p.y + static_cast<size_t>(row0) * p.N + t.n0;
#pragma unroll 1
        for (int c0 = 0; c0 < C::N; c0 += 32) {
          uint32_t v[32];
          tc::tmem_ld32(ta + c0, v);
          if (c0 + 32 == C::N) hand_back(ac);
          if (t.n0 + c0 >= p.N) continue;
          uint4 o[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (p.bias != nullptr && t.n0 + c0 + 8 * c < p.N) {
              const uint4 bb = *reinterpret_cast<const uint4*>(p.bias + t.n0 + c0 + 8 * c);
              b[0] = bf16_lo(bb.x), b[1] = bf16_hi(bb.x), b[2] = bf16_lo(bb.y), b[3] = bf16_hi(bb.y);
              b[4] = bf16_lo(bb.z), b[5] = bf16_hi(bb.z), b[6] = bf16_lo(bb.w), b[7] = bf16_hi(bb.w);
            }
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = fmaf(__uint_as_float(v[8 * c + j]), alpha, b[j]);
            o[c] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                              pack_bf16x2(f[6], f[7]));
          }
          rows_out(buf, o, [&](int r, int c, const uint4& x) {
            if (row0 + r < t.row_end && t.n0 + c0 + 8 * c < p.N)   // N is a multiple of 8
              *reinterpret_cast<uint4*>(yp + static_cast<size_t>(r) * p.N + c0 + 8 * c) = x;
          });
        }
      } else {
        const int o = 32 * warp + lane, n = t.n0 + o, valid = t.row_end - t.row0;
        if (p.split > 1) {
          float* mine = reinterpret_cast<float*>(ring) + o;   // every copy has landed and every MMA is done
#pragma unroll 1
          for (int c0 = 0; c0 < C::N && c0 < valid; c0 += 16) {
            uint32_t v[16];
            tc::tmem_ld16_async(ta + c0, v);
            tc::tmem_wait_ld(v);
#pragma unroll
            for (int j = 0; j < 16; ++j) mine[(c0 + j) * 128] = __uint_as_float(v[j]);   // past the last token too
          }
        } else {
          const float b = p.bias != nullptr && n < p.N ? __uint_as_float(static_cast<uint32_t>(p.bias[n]) << 16) : 0.f;
          uint16_t* yp = p.y + static_cast<size_t>(t.row0) * p.N + n;
#pragma unroll 1
          for (int c0 = 0; c0 < C::N && c0 < valid; c0 += 16) {
            uint32_t v[16];
            tc::tmem_ld16_async(ta + c0, v);
            tc::tmem_wait_ld(v);
            if (n < p.N) {
#pragma unroll
              for (int j = 0; j < 16; ++j, yp += p.N)
                if (c0 + j < valid) *yp = static_cast<uint16_t>(f32_to_bf16_bits(fmaf(__uint_as_float(v[j]), alpha, b)));
            }
          }
        }
        hand_back(ac);
      }
      if (++ac == C::ACCS) ac = 0, aph ^= 1;
    }
  }
  __syncwarp();

  if constexpr (kForm == kStream) {
    if (p.split > 1) {
      // One item per cluster: CTA r adds the parts of tokens r, r + split, ... in the order
      // of the parts. A warp takes a token, 4 outputs a lane.
      cluster_arrive();
      cluster_wait();
      int e = 0;
      Tile t;
      if (decode(seg, first, X, W, starts, t, e) && !*abort_flag) {
        const int n = t.n0 + 4 * lane;
        if (n < p.N) {
          const float alpha = (p.x_global != nullptr ? __ldcg(p.x_global) : 1.f) * (p.w_global != nullptr ? __ldcg(p.w_global) : 1.f);
          float b[4] = {0.f, 0.f, 0.f, 0.f};
          if (p.bias != nullptr) {
            const uint2 bb = *reinterpret_cast<const uint2*>(p.bias + n);
            b[0] = bf16_lo(bb.x), b[1] = bf16_hi(bb.x), b[2] = bf16_lo(bb.y), b[3] = bf16_hi(bb.y);
          }
          for (int j = part + warp * p.split; j < t.row_end - t.row0; j += C::THREADS / 32 * p.split) {
            const uint32_t at = smem_addr(ring) + (j * 128 + 4 * lane) * 4;
            float4 v[kMaxSplit];
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r)
              if (r < p.split) v[r] = ld_cluster_f32x4(at, r);
            float4 s = v[0];
#pragma unroll
            for (int r = 1; r < kMaxSplit; ++r)
              if (r < p.split) s.x += v[r].x, s.y += v[r].y, s.z += v[r].z, s.w += v[r].w;
            *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(t.row0 + j) * p.N + n) =
                make_uint2(pack_bf16x2(fmaf(s.x, alpha, b[0]), fmaf(s.y, alpha, b[1])),
                           pack_bf16x2(fmaf(s.z, alpha, b[2]), fmaf(s.w, alpha, b[3])));
          }
        }
      }
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    }
  }

  if (*abort_flag) {   // let copies and MMAs in flight land before the shared memory goes away
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Row tiles of `per` rows that R rows in E segments can need at most.
int64_t row_tiles(const Fp4Args& a, int per) {
  const int64_t whole = (a.R + per - 1) / per;
  return a.expert_offsets == nullptr ? whole : (a.R < whole + a.E ? a.R : whole + a.E);
}

template <int W, int X, bool kNv, Form kForm, bool kQuant = false>
cudaError_t run(const Fp4Args& a, Params& p, cudaStream_t s) {
  using C = Shape<W, X, kNv, kForm, kQuant>;
  cudaError_t e = kQuant ? cudaSuccess : encode(&p.tm_x, a.qx, a.K / 2, a.R, 0, X);
  if (e == cudaSuccess) e = encode(&p.tm_w, a.qweight, a.K / 2, a.N, a.E, W);
  if (e == cudaSuccess && p.tma_scales && !kQuant) e = encode(&p.tm_xs, a.x_scale, p.SB, a.R, 0, X, 1, 32);
  if (e == cudaSuccess && p.tma_scales) e = encode(&p.tm_ws, a.w_scale, p.SB, a.N, a.E, W, 1, 32);
  if (e != cudaSuccess) return e;
  p.n_tiles = static_cast<int>((a.N + W - 1) / W);
  const int64_t items = row_tiles(a, X) * p.n_tiles;
  if (items > kMaxItems) return cudaErrorInvalidConfiguration;
  p.items = static_cast<int>(items);
  p.split = 1;
  const int64_t slots = static_cast<int64_t>(current_sm_count()) * C::CTAS;
  if (kForm == kStream && a.expert_offsets == nullptr)
    for (int n = kMaxSplit; n > 1 && p.split == 1; --n)
      if (p.KS >= 2 * n && items <= clusters_held(n, X > 16 ? 1 : C::CTAS)) p.split = n;
  const int64_t grid = p.split > 1 ? items * p.split : (items < slots ? items : slots);
  return start<fp4_kernel<W, X, kNv, kForm, kQuant>>(p, grid, C::THREADS, C::SMEM, p.split, s);
}

template <bool kNv>
cudaError_t launch(const Fp4Args& a, Params& p, cudaStream_t s) {
  const bool experts = a.expert_offsets != nullptr;
  // Experts' rows on average, as only the device knows each one's. Where they are uneven the tile form may be a little
  // better: 256 tokens, half of whose 8 choices are the same four of 64 experts, N 2816, K 2048 nvfp4 45.7 us, 43.6 in tiles.
  const int64_t rows = (a.R + a.E - 1) / a.E;
  if (a.x != nullptr) return run<128, 16, kNv, kStream, true>(a, p, s);
  if (rows <= 16) return run<128, 16, kNv, kStream>(a, p, s);
  if (rows <= 32) return run<128, 32, kNv, kStream>(a, p, s);
  if (rows <= 64) return run<128, 64, kNv, kStream>(a, p, s);
  if (!experts) {
    const int64_t sms = current_sm_count();
    auto tiles = [&](int64_t x, int64_t w) { return (a.R + x - 1) / x * ((a.N + w - 1) / w); };
    // Clusters that cut k where the weights' tiles are few: 300 x 2048 x 8192 nvfp4 10.4 us, tiles
    // 14.0. Without room for three parts tiles are as good (517 x 4096 x 4096 9.6 against 12.0).
    if (rows <= 128 || 3 * tiles(128, 128) <= sms) return run<128, 128, kNv, kStream>(a, p, s);
  }
  return run<192, 128, kNv, kTile>(a, p, s);
}

}  // namespace

bool fp4_fuses(int64_t R, bool experts) { return !experts && R <= kFuseRows; }

cudaError_t launch_fp4(const Fp4Args& a, cudaStream_t s) {
  Params p;
  memset(&p, 0, sizeof(p));
  p.x = static_cast<const uint4*>(a.x);
  p.x_f16 = a.x_f16;
  p.x_wide = (reinterpret_cast<uintptr_t>(a.x) & 31) == 0;
  p.x_scale = static_cast<const uint8_t*>(a.x_scale);
  p.w_scale = static_cast<const uint8_t*>(a.w_scale);
  p.x_global = a.x_global;
  p.w_global = a.w_global;
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.y = static_cast<uint16_t*>(a.y);
  p.offsets = a.expert_offsets;
  p.E = a.E;
  p.rows = static_cast<int>(a.R);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.SB = static_cast<int>(a.K / fp4_block(a.nv));
  p.KS = static_cast<int>((a.K + kStageK - 1) / kStageK);
  // rows of scales that TMA takes; words one by one otherwise
  p.tma_scales = p.SB % 16 == 0 && ((reinterpret_cast<uintptr_t>(a.x_scale) | reinterpret_cast<uintptr_t>(a.w_scale)) & 15) == 0;
  p.status = a.status;
  return a.nv ? launch<true>(a, p, s) : launch<false>(a, p, s);
}

}  // namespace w4
