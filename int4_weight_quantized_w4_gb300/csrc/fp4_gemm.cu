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
// memory, as checkpoints hold them; the MMA wants them in tensor memory with 128 rows'
// words in four columns. Scale warps copy a row's words of a stage (16 bytes nvfp4, 8
// mxfp4) asynchronously to their places in shared memory, and the MMA warp sends each
// 512-byte atom on to tensor memory ahead of the MMAs that use it.
//
// Two forms:
//  * stream (few rows): weights on the MMA's 128 rows, NT tokens on its columns; dense
//    products share a tile's k among the CTAs of a cluster. Bound by the weight bytes.
//  * tile (many rows): 128 tokens on the MMA's rows, 192 outputs on its columns, with
//    two accumulators, so that the MMAs of a tile run while the one before leaves.
//
// Both are launched as programmatic dependents and let their own dependents go early: the
// weights and their scales start while the kernels before finish, everything else waits.
#include <cstring>

#include "common.cuh"
#include "launch.h"
#include "tc.cuh"
#include "tiles.cuh"

namespace w4 {
namespace {

constexpr int kStageK = 256;                  // columns of a stage
constexpr int kStageBytes = kStageK / 2;

struct Params {
  CUtensorMap tm_x;        // codes [rows, K/2 bytes]
  CUtensorMap tm_w;        // codes [E, N, K/2 bytes]
  const uint8_t* x_scale;  // [rows, SB]
  const uint8_t* w_scale;  // [E, N, SB]
  const float* x_global;   // or null
  const float* w_global;   // [E], or null
  const uint16_t* bias;    // bf16 [N] or null
  uint16_t* y;             // bf16 [rows, N]
  const int32_t* offsets;  // [E + 1], or null (dense: one segment of all rows)
  int E, rows, N, K, SB, KS, n_tiles;   // SB: scale bytes a row, KS: stages over k
  int split;               // stream form, dense: parts of the stages, one per CTA of a cluster
  int items;
  unsigned int* status;
};

// Rows [a, b) of expert e; a segment outside [0, rows) counts as clipped. The offsets
// are read from L2, where the kernel that wrote them left them.
W4_DEV void seg_bounds(const Params& p, int e, int& a, int& b) {
  a = max(__ldcg(p.offsets + e), 0);
  b = min(__ldcg(p.offsets + e + 1), p.rows);
}

// W: weight rows of a tile, X: tokens of a tile; the one on the MMA's rows is 128.
template <int W, int X, bool kNv, bool kTile>
struct Shape {
  static constexpr int WORDS = kNv ? 4 : 2;                    // 32-bit scale words of a row's stage
  static constexpr int N = kTile ? W : X;                      // MMA columns
  static constexpr int ATOMS_W = (W + 127) / 128, ATOMS_X = (X + 127) / 128;
  static constexpr int W_BYTES = W * kStageBytes, X_BYTES = X * kStageBytes;
  static constexpr int SW_BYTES = ATOMS_W * WORDS * 512, SX_BYTES = ATOMS_X * WORDS * 512;
  static constexpr int STAGE = W_BYTES + X_BYTES;
  static constexpr int SSTAGE = SW_BYTES + SX_BYTES;
  static constexpr int CTAS = kTile || X > 64 ? 1 : 2;         // resident per SM
  static constexpr int STAGES = CTAS == 2 ? (X == 64 ? 3 : 4) : kTile ? 4 : 5;
  static constexpr int AHEAD = STAGES - 2;                     // stages of scale copies in flight (reported before the ring is full)
  static constexpr int ACCS = 2;
  static constexpr int S_COLS = 4 * WORDS * (ATOMS_W + ATOMS_X);   // tensor memory columns of a stage's scales
  static constexpr int USED = ACCS * N + 2 * S_COLS;
  static constexpr int TMEM_COLS = USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
  // warps: 4 epilogue, the MMA issuer, then those that copy weights and their scales, then the activations'
  static constexpr int WW = W / 32 > 4 ? 4 : W / 32, XW = X / 32 > 4 ? 4 : X < 32 ? 1 : X / 32;
  static constexpr int THREADS = 32 * (5 + WW + XW);
  static constexpr int OUT = kTile ? 4 * 2048 : 0;
  static constexpr int SMEM = STAGES * (STAGE + SSTAGE) + OUT + 256 + (kMaxExperts + 1 + 16 + 3) / 4 * 16 + 1024;
  static_assert(USED <= 512 && CTAS * TMEM_COLS <= 512, "tensor memory");
  static_assert(SMEM <= 232448 && CTAS * SMEM + CTAS * 1024 <= 233472, "shared memory");
  static_assert((2 * STAGES + 2 * ACCS) * 8 + 8 <= 256, "barriers");
  static_assert(STAGE % 1024 == 0 && W_BYTES % 1024 == 0, "swizzle atoms");
  static_assert(kTile || X * 512 <= STAGES * STAGE, "part sums of a cluster fit the ring");
};

// Scale words of `ROWS` rows from row0 on (those below `valid` exist), stage ks, by warps
// of which this one is number `w` of `kWarps`: word j of row r to atom j * ATOMS + r / 128,
// at 16 (r % 32) + 4 (r / 32 % 4). Words past the row's end are zeros.
template <int ROWS, int WORDS, int kWarps>
W4_DEV void load_scales(uint32_t to, const uint8_t* src, int SB, int ks, int valid, int w) {
  constexpr int ATOMS = (ROWS + 127) / 128;
  const int lane = threadIdx.x & 31;
  const int at = ks * WORDS * 4;
#pragma unroll
  for (int r0 = 0; r0 < ROWS; r0 += 32 * kWarps) {
    const int r = r0 + 32 * w + lane;
    if (r0 + 32 * kWarps <= ROWS || r < ROWS) {
      const uint32_t d = to + (r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
      const bool in = r < valid;
      const uint8_t* s = src + static_cast<size_t>(in ? r : 0) * SB + at;
#pragma unroll
      for (int j = 0; j < WORDS; ++j) {
        const bool word = in && at + 4 * j < SB;
        tc::copy4_async(d + j * ATOMS * 512, word ? s + 4 * j : src, word);
      }
    }
  }
}

template <int W, int X, bool kNv, bool kTile>
__global__ void __launch_bounds__(Shape<W, X, kNv, kTile>::THREADS, Shape<W, X, kNv, kTile>::CTAS)
fp4_kernel(const __grid_constant__ Params p) {
  using C = Shape<W, X, kNv, kTile>;
  constexpr int kMma = 4, kW0 = 5, kX0 = 5 + C::WW;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;                               // per stage: weights, activations
  uint8_t* scales = ring + C::STAGES * C::STAGE;      // per stage: weights', activations'
  uint4* out_base = reinterpret_cast<uint4*>(scales + C::STAGES * C::SSTAGE);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(out_base) + C::OUT);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + C::ACCS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_empty + C::ACCS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int32_t* starts = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(full) + 256);
  int32_t* warp_sum = starts + kMaxExperts + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 2 + C::WW + C::XW);   // two copies by TMA, the scale warps
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::ACCS; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMma) tc::tmem_alloc(tmem_holder, C::TMEM_COLS);
  if (warp == kW0 && lane == 0) tc::prefetch_tmap(&p.tm_w);
  if (warp == kX0 && lane == 0) tc::prefetch_tmap(&p.tm_x);
  if (p.offsets != nullptr) {
    grid_dependency_wait();   // the routing may be running still
    tile_starts<C::THREADS>(p, X, starts, warp_sum);
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

  if (warp >= kW0) {
    // Copies of weights (kW0 ..) or activations (kX0 ..): a whole warp walks the ring, its
    // lanes copy scales, lane 0 of the first warp the operand. A stage's scales are
    // reported full AHEAD stages later, when their copies have landed.
    const bool mine_w = warp < kX0;
    const int w = mine_w ? warp - kW0 : warp - kX0;
    int st = 0, ph = 1, e = 0, g = 0;
    bool ok = true, waited = false;
    Tile t;
    if (!mine_w) grid_dependency_wait();   // the codes come from the kernel before
    auto landed = [&](int stage) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[stage]);
    };
    for (int it = first; ok && it < p.items && decode(p, it, X, W, starts, t, e); it += step)
      for (int ks = ks0; ks < ks1; ++ks) {
        if (mine_w && ph == 0 && !waited) {   // the ring is full, and is emptied only after the kernels before
          grid_dependency_wait();
          waited = true;
        }
        if (!(ok = wait_warp(&empty[st], ph, abort_flag, p.status))) break;
        uint8_t* to = ring + st * C::STAGE;
        const uint32_t sc = smem_addr(scales + st * C::SSTAGE);
        if (mine_w) {
          if (w == 0 && lane == 0) {
            mbar_arrive_expect_tx(&full[st], C::W_BYTES);
            tc::tma_load_3d(to, &p.tm_w, &full[st], ks * kStageBytes, t.n0, t.expert);
          }
          load_scales<W, C::WORDS, C::WW>(sc, p.w_scale + (static_cast<size_t>(t.expert) * p.N + t.n0) * p.SB, p.SB, ks,
                                          p.N - t.n0, w);
        } else {
          if (w == 0 && lane == 0) {
            mbar_arrive_expect_tx(&full[st], C::X_BYTES);
            tc::tma_load_2d(to + C::W_BYTES, &p.tm_x, &full[st], ks * kStageBytes, t.row0);
          }
          load_scales<X, C::WORDS, C::XW>(sc + C::SW_BYTES, p.x_scale + static_cast<size_t>(t.row0) * p.SB, p.SB, ks,
                                          t.row_end - t.row0, w);
        }
        tc::copy_async_commit();
        if (g >= C::AHEAD) {
          tc::copy_async_wait<C::AHEAD>();
          landed(st >= C::AHEAD ? st - C::AHEAD : st - C::AHEAD + C::STAGES);
        }
        ++g;
        if (++st == C::STAGES) st = 0, ph ^= 1;
      }
    tc::copy_async_wait<0>();
    if (ok)
      for (int i = g < C::AHEAD ? g : C::AHEAD; i > 0; --i) landed(st >= i ? st - i : st - i + C::STAGES);
  } else if (warp == kMma) {
    grid_dependency_wait();
    constexpr uint32_t idesc = tc::idesc_fp4<kNv>(128, C::N);
    const bool leader = elect_one();
    const uint64_t wd0 = tc::sdesc_sw128(smem_addr(ring)), xd0 = wd0 + (C::W_BYTES >> 4);
    const uint64_t sd0 = tc::sdesc_scales(smem_addr(scales));
    int st = 0, ph = 0, ac = 0, aph = 1, e = 0, buf = 0;
    bool ok = true;
    Tile t;
    for (int it = first; ok && it < p.items && decode(p, it, X, W, starts, t, e); it += step) {
      if (!(ok = wait_warp(&acc_empty[ac], aph, abort_flag, p.status))) break;
      for (int ks = ks0; ks < ks1; ++ks) {
        if (!(ok = wait_warp(&full[st], ph, abort_flag, p.status))) break;
        tc::fence_after_sync();
        if (leader) {
          // weights' scales, then the activations': [word][atom][4 columns] each
          const uint32_t sw = tmem + C::ACCS * C::N + buf * C::S_COLS, sx = sw + 4 * C::WORDS * C::ATOMS_W;
          const uint64_t sd = sd0 + static_cast<uint64_t>((st * C::SSTAGE) >> 4);
#pragma unroll
          for (int i = 0; i < C::WORDS * (C::ATOMS_W + C::ATOMS_X); ++i) tc::copy_scales(sw + 4 * i, sd + 32 * i);
          const uint64_t wd = wd0 + static_cast<uint64_t>((st * C::STAGE) >> 4);
          const uint64_t xd = xd0 + static_cast<uint64_t>((st * C::STAGE) >> 4);
          const int left = p.K - ks * kStageK;
#pragma unroll
          for (int j = 0; j < 4; ++j) {   // 64 columns, 32 bytes, at a time
            if (64 * j >= left) break;
            const int word = kNv ? j : j >> 1;
            const uint32_t id = idesc | (kNv || !(j & 1) ? 0u : (2u << 29) | (2u << 4));
            const uint32_t fw = sw + 4 * C::ATOMS_W * word, fx = sx + 4 * C::ATOMS_X * word;
            const uint32_t acc = ks > ks0 || j > 0 ? 1u : 0u;
            if constexpr (kTile)
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
    for (int it = first; ok && it < p.items && decode(p, it, X, W, starts, t, e); it += step) {
      const float alpha = p.w_global != nullptr ? gx * __ldcg(p.w_global + t.expert) : gx;
      if (!(ok = wait_warp(&acc_full[ac], aph, abort_flag, p.status))) break;
      tc::fence_after_sync();
      const uint32_t ta = tmem + (static_cast<uint32_t>(32 * warp) << 16) + ac * C::N;
      if constexpr (kTile) {
        const int row0 = t.row0 + 32 * warp;
        uint4* buf = out_base + warp * 128;
        uint16_t* yp = p.y + static_cast<size_t>(row0) * p.N + t.n0;
#pragma unroll 1
        for (int c0 = 0; c0 < C::N; c0 += 32) {
          uint32_t v[32];
          tc::tmem_ld32(ta + c0, v);
          if (c0 + 32 == C::N) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[ac]);
          }
          if (t.n0 + c0 < p.N) {
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
        }
      } else {
        const int o = 32 * warp + lane, n = t.n0 + o, valid = t.row_end - t.row0;
        const float b = p.split == 1 && p.bias != nullptr && n < p.N ? __uint_as_float(static_cast<uint32_t>(p.bias[n]) << 16) : 0.f;
        float* mine = reinterpret_cast<float*>(ring);   // split: every copy has landed and every MMA is done
        uint16_t* yp = p.y + static_cast<size_t>(t.row0) * p.N + n;
#pragma unroll 1
        for (int c0 = 0; c0 < C::N; c0 += 16) {
          if (c0 >= valid) break;
          uint32_t v[16];
          tc::tmem_ld16_async(ta + c0, v);
          tc::tmem_wait_ld(v);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (c0 + j >= valid) break;
            if (p.split > 1)
              mine[(c0 + j) * 128 + o] = __uint_as_float(v[j]);
            else if (n < p.N)
              yp[static_cast<size_t>(c0 + j) * p.N] = static_cast<uint16_t>(f32_to_bf16_bits(fmaf(__uint_as_float(v[j]), alpha, b)));
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[ac]);
      }
      if (++ac == C::ACCS) ac = 0, aph ^= 1;
    }
  }
  __syncwarp();

  if constexpr (!kTile) {
    if (p.split > 1) {
      // One item per cluster: CTA r adds the parts of tokens r, r + split, ... in the order
      // of the parts. A warp takes a token, 4 outputs a lane.
      cluster_arrive();
      cluster_wait();
      int e = 0;
      Tile t;
      if (decode(p, first, X, W, starts, t, e) && !*abort_flag) {
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

template <int W, int X, bool kNv, bool kTile>
cudaError_t run(const Fp4Args& a, Params& p, cudaStream_t s) {
  using C = Shape<W, X, kNv, kTile>;
  cudaError_t e = encode(&p.tm_x, a.qx, a.K / 2, a.R, 0, X);
  if (e != cudaSuccess) return e;
  e = encode(&p.tm_w, a.qweight, a.K / 2, a.N, a.E, W);
  if (e != cudaSuccess) return e;
  p.n_tiles = static_cast<int>((a.N + W - 1) / W);
  const int64_t items = row_tiles(a, X) * p.n_tiles;
  if (items > kMaxItems) return cudaErrorInvalidConfiguration;
  p.items = static_cast<int>(items);
  const int64_t slots = static_cast<int64_t>(current_sm_count()) * C::CTAS;
  p.split = 1;
  if (!kTile && a.expert_offsets == nullptr)
    for (int n = kMaxSplit; n > 1 && p.split == 1; --n)
      if (p.KS >= 2 * n && items <= clusters_held(n, C::CTAS)) p.split = n;
  const int64_t grid = p.split > 1 ? items * p.split : (items < slots ? items : slots);
  return start<fp4_kernel<W, X, kNv, kTile>>(p, grid, C::THREADS, C::SMEM, p.split, s);
}

template <bool kNv>
cudaError_t launch(const Fp4Args& a, Params& p, cudaStream_t s) {
  const bool experts = a.expert_offsets != nullptr;
  const int64_t rows = (a.R + a.E - 1) / a.E;
  if (rows <= 16) return run<128, 16, kNv, false>(a, p, s);
  if (rows <= 32) return run<128, 32, kNv, false>(a, p, s);
  if (rows <= 64) return run<128, 64, kNv, false>(a, p, s);
  if (!experts && rows <= 128) return run<128, 128, kNv, false>(a, p, s);
  return run<192, 128, kNv, true>(a, p, s);
}

}  // namespace

cudaError_t launch_fp4(const Fp4Args& a, cudaStream_t s) {
  Params p;
  memset(&p, 0, sizeof(p));
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
  p.status = a.status;
  return a.nv ? launch<true>(a, p, s) : launch<false>(a, p, s);
}

}  // namespace w4
