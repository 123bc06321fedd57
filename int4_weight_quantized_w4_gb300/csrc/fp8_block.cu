// The fp8 block-scaled product on the 5th-generation tensor cores (tcgen05,
// kind::f8f6f4, sm_103a), dense and over expert segments of rows:
//
//   y[r, n] = bf16( sum_b sx[r, b] sw[n / 128, b] P[r, b, n] + bias[n] ),
//   P[r, b, n] = sum_{k in block b} q[r, k] w[n, k],
//
// q, w e4m3, blocks of 128 along k, fp32 scales. P is accumulated in fp32 by
// the tensor core, one accumulation per block, because sx and sw are arbitrary
// fp32 numbers; the sum over blocks is an fp32 FMA per element in registers.
//
// Two forms:
//  * stream (few rows an expert or call): weights on the MMA's 128 rows (TMEM
//    lane = output), NT tokens on its columns. Bound by the weight bytes (0.92 of copy
//    bandwidth at 1 x 131072 x 2048, 43 us) and some 3.5 us a call (0.67 at 1 x
//    14336 x 4096, 12.9 us). For up to kFuseRows dense rows the kernel quantizes 16-bit
//    activations itself.
//  * tile (many rows): 128 tokens on the MMA's rows, 256 outputs on its columns,
//    so that one scale sx * sw serves a thread's whole column strip. Bound by the
//    hand-over and drain of one accumulator per block: about 920 cycles a block,
//    of which the barriers' round trip takes some 450, the FMAs 290 (256 are their
//    issue time) and what shows of the reads of tensor memory 100 (256 by themselves),
//    where its MMAs take 512 and its 48 KB of operands 860; and by 1.7 us a tile for
//    its outputs, in which the MMAs stand still. 4096 x 11008 x 4096 takes 165 us with
//    its quantizer, and 153 alone on an idle card, 2.4 PFLOP/s.
//
// Times in this file are GPU times of a call in a CUDA graph of calls on inputs that
// rotate past L2; a pair is the two sides measured in one run. Large products vary by
// some 5% with what the card's power limit leaves, and a chain of calls from Python is
// within 10% of a graph (173 to 176 us at 4096 x 11008 x 4096).
//
// Both are launched as programmatic dependents and let their own dependents go
// early: the copies of weights start while the kernels before finish, everything
// else (activations, scales, bias, y) waits for them (griddepcontrol.wait), and so do the expert offsets
// unless the one before is the row quantizer, which starts this one only when all
// before it are done.
#include <atomic>
#include <cstring>

#include "common.cuh"
#include "launch.h"
#include "tc.cuh"
#include "tiles.cuh"

namespace w4 {
namespace {

constexpr int kBlk = 128;                     // k and weight rows per scale
// Up to this many dense rows the stream form quantizes: one launch less (fused / not:
// 1 x 4096 x 4096 6.3 / 7.1 us, 8 x 4096 x 4096 7.0 / 7.6, 8 x 14336 x 4096 14.3 / 14.4). Every
// CTA quantizes them again, so that at 16 rows the order turns (8.5 / 8.0).
constexpr int kFuseRows = 8;

struct Params {
  CUtensorMap tm_x;        // e4m3 codes [rows, K] (unused where the kernel quantizes)
  CUtensorMap tm_w;        // e4m3 codes [E, N, K]
  const float* x_scale;    // [rows, KB]
  const uint4* x;          // 16-bit activations [rows, K] to quantize, or null
  bool x_f16;
  const float* w_scale;    // [E, NB, KB]
  const uint16_t* bias;    // bf16 [N] or null
  uint16_t* y;             // bf16 [rows, N]
  const int32_t* offsets;  // [E + 1], or null (dense: one segment of all rows)
  bool offsets_ready;      // whatever writes them is done when this kernel starts
  int E, rows, N, K, KB, NB, n_tiles;
  int split;               // stream form, dense: parts of the k blocks, one per CTA of a cluster
  int items;               // upper bound of (row tile, n tile) pairs, or of the tile form's work items
  // tile form, dense: items 0 .. full - 1 are whole tiles; item full + j is part
  // j % parts of the k blocks of tile full + j / parts, summed into part_sums
  int full;
  int parts;
  float* part_sums;        // fp32 [tile - full][part][TM][TN]
  unsigned int* status;
};

// Rows [a, b) of expert e; a segment outside [0, rows) counts as clipped. The offsets
// are read from L2, where the kernel that wrote them left them: with offsets_ready this
// one has not waited for the kernels before yet.
W4_DEV void seg_bounds(const Params& p, int e, int& a, int& b) {
  a = max(__ldcg(p.offsets + e), 0);
  b = min(__ldcg(p.offsets + e + 1), p.rows);
}

// Where part `i` of `n` of KB blocks starts (KB, n below 2^15 and 2^5, or n = 1).
W4_DEV int part_start(int KB, int i, int n) { return n == 1 ? i * KB : KB * i / n; }

// e4m3 x e4m3, fp32 accumulator, both operands K-major: format codes 0.
// One block of 128 k: four MMAs of 32 k, 32 bytes apart in the swizzle row.
W4_DEV void mma_block(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
  for (int j = 0; j < 4; ++j) tc::mma_f8(d, a + 2 * j, b + 2 * j, idesc, j > 0 ? 1u : 0u);
}

// ---------------------------------------------------------------------------
// stream form
// ---------------------------------------------------------------------------

template <int NT, bool kQuant>
struct Stream {
  static constexpr int A_BYTES = kBlk * 128;             // 128 outputs x 128 k
  static constexpr int B_BYTES = NT * 128;               // NT tokens x 128 k
  static constexpr int CTAS = NT <= 64 ? 2 : 1;          // resident per SM
  static constexpr int STAGES = NT <= 32 ? 5 : NT == 64 ? 4 : 6;
  static constexpr int TMEM_COLS = CTAS == 2 ? 256 : 512;
  static constexpr int ACCS = TMEM_COLS / NT > 8 ? 8 : TMEM_COLS / NT;
  static constexpr int SC_PER = kQuant ? 1 : 4;          // blocks per scale slot (x NT tokens)
  static constexpr int SC_SLOTS = kQuant ? 8 : 4;
  static constexpr int SC_ROW = kQuant ? NT : NT + 8;    // 8 rows x 4 blocks of a slot lie in 32 banks
  static constexpr int SC_BYTES = SC_SLOTS * SC_PER * SC_ROW * 4;
  static constexpr int THREADS = kQuant ? 320 : 256;
  static constexpr int SMEM = STAGES * (A_BYTES + B_BYTES) + SC_BYTES + 512 + (kMaxExperts + 1 + 10 + 5) / 4 * 16 + 1024;
};
static_assert(Stream<16, true>::SMEM * 2 + 2048 <= 233472 && Stream<32, false>::SMEM * 2 + 2048 <= 233472 && Stream<64, false>::SMEM * 2 + 2048 <= 233472 &&
                  Stream<128, false>::SMEM <= 232448,
              "shared memory per SM");

// Warps 0-3 epilogue (warp w: TMEM lanes 32 w, outputs n0 + 32 w + lane), 4
// weight copies, 5 MMA issuer and TMEM owner; then 6 activation copies and 7
// scales, or (kQuant: dense, one row tile) 6-9 quantizers of alternate blocks.
constexpr int kSWarpA = 4, kSWarpMma = 5, kSWarpB = 6, kSWarpScale = 7;
constexpr int kQuantWarps = 4;
// A quantizer sees every fourth phase of the ring barriers it waits on. Before its
// block g it waited for block g - 4 - S to be done (S slots); with S >= 4 that is
// block g - 2 S or a later one, so a parity names one phase.
static_assert(Stream<16, true>::STAGES >= kQuantWarps && Stream<16, true>::SC_SLOTS >= kQuantWarps, "see above");

template <int NT, bool kQuant>
__global__ void __launch_bounds__(Stream<NT, kQuant>::THREADS, Stream<NT, kQuant>::CTAS) stream_kernel(const __grid_constant__ Params p) {
  using C = Stream<NT, kQuant>;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* a_base = smem;
  uint8_t* b_base = a_base + C::STAGES * C::A_BYTES;
  float* sc_base = reinterpret_cast<float*>(b_base + C::STAGES * C::B_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sc_base) + C::SC_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + C::ACCS;
  uint64_t* sc_full = acc_empty + C::ACCS;
  uint64_t* sc_empty = sc_full + C::SC_SLOTS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sc_empty + C::SC_SLOTS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int32_t* starts = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(full) + 512);
  int32_t* warp_sum = starts + kMaxExperts + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::ACCS; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    for (int i = 0; i < C::SC_SLOTS; ++i) {
      mbar_init(&sc_full[i], 1);
      mbar_init(&sc_empty[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kSWarpMma) tc::tmem_alloc(tmem_holder, C::TMEM_COLS);
  if (warp == kSWarpA && lane == 0) tc::prefetch_tmap(&p.tm_w);
  if (!kQuant && warp == kSWarpB && lane == 0) tc::prefetch_tmap(&p.tm_x);
  if (p.offsets != nullptr) {
    if (!p.offsets_ready) grid_dependency_wait();   // the routing may be running still
    tile_starts<C::THREADS>(p, NT, starts, warp_sum);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  launch_dependents();
  const uint32_t tmem = *tmem_holder;

  // this CTA's part of the k blocks (the same for every item)
  const int part = p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int kb0 = part_start(p.KB, part, p.split), kb1 = part_start(p.KB, part + 1, p.split);
  const int first = blockIdx.x / p.split, step = gridDim.x / p.split;

  if (warp == kSWarpA) {
    if (lane == 0) {
      int st = 0, ph = 1, e = 0;
      bool ok = true, waited = false;
      Tile t;
      for (int it = first; ok && it < p.items && decode(p, it, NT, kBlk, starts, t, e); it += step)
        for (int kb = kb0; kb < kb1; ++kb) {
          if (ph == 0 && !waited) {   // the ring is full, and is emptied only after the kernels before
            grid_dependency_wait();
            waited = true;
          }
          if (!(ok = tc::wait(&empty[st], ph, abort_flag, p.status, kWaitNs))) break;
          mbar_arrive_expect_tx(&full[st], C::A_BYTES);
          tc::tma_load_3d(a_base + st * C::A_BYTES, &p.tm_w, &full[st], kb * kBlk, t.n0, t.expert);
          if (++st == C::STAGES) st = 0, ph ^= 1;
        }
    }
  } else if (kQuant && warp >= kSWarpB) {
    // Quantizer w takes blocks w, w + 4, ... of this CTA's sequence: half-warp h the
    // rows h + 2 u, all of a block's at once (one or two rows by a shorter path: at 1
    // x 14336 x 4096 12.8 us against 13.4). The chunks of its next block are loaded
    // as soon as this one's are used.
    if constexpr (kQuant) {
      static_assert(kFuseRows == 8, "four rows a half-warp");
      const int h = lane >> 4, l = lane & 15;
      const int K8 = p.K >> 3, nkb = kb1 - kb0;
      const int total = first < p.items ? (p.items - first + step - 1) / step * nkb : 0;
      auto load = [&](int g, int r) {
        const int c = (kb0 + g % nkb) * 16 + l;
        return r < p.rows && c < K8 && g < total ? p.x[static_cast<size_t>(r) * K8 + c] : make_uint4(0, 0, 0, 0);
      };
      uint4 x[4];
      grid_dependency_wait();   // x comes from the kernel before
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = load(warp - kSWarpB, h + 2 * u);
      for (int g = warp - kSWarpB; g < total; g += kQuantWarps) {
        const int kb = kb0 + g % nkb;
        const int nt = (first + g / nkb * step) % p.n_tiles;
        const float sw = p.w_scale[static_cast<size_t>(nt) * p.KB + kb];
        const int st = g % C::STAGES, sl = g % C::SC_SLOTS;
        if (!wait_warp(&empty[st], ((g / C::STAGES) & 1) ^ 1, abort_flag, p.status)) break;
        if (!wait_warp(&sc_empty[sl], ((g / C::SC_SLOTS) & 1) ^ 1, abort_flag, p.status)) break;
        uint8_t* to = b_base + st * C::B_BYTES + (l & 1) * 8;
        float* sc = sc_base + sl * NT;
        // a row past the last one fills a column that is never stored
        if (p.rows <= 2) {
          uint2 code;
          float s;
          if (p.x_f16)
            quant_block_half_warp<true>(x[0], code, s);
          else
            quant_block_half_warp<false>(x[0], code, s);
          x[0] = load(g + kQuantWarps, h);
          *reinterpret_cast<uint2*>(to + h * 128 + (((l >> 1) ^ h) << 4)) = code;
          if (l == 0) sc[h] = s * sw;
        } else {
          uint2 code[4];
          const float s = p.x_f16 ? quant_blocks4<true>(x, code) : quant_blocks4<false>(x, code);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = h + 2 * u;
            x[u] = load(g + kQuantWarps, r);
            *reinterpret_cast<uint2*>(to + r * 128 + (((l >> 1) ^ r) << 4)) = code[u];
          }
          if (l < 4) sc[h + 2 * l] = s * sw;
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[st]);
          mbar_arrive(&sc_full[sl]);
        }
      }
    }
  } else if (warp == kSWarpB) {
    if (lane == 0) {
      grid_dependency_wait();   // the codes come from the kernel before
      int st = 0, ph = 1, e = 0;
      bool ok = true;
      Tile t;
      for (int it = first; ok && it < p.items && decode(p, it, NT, kBlk, starts, t, e); it += step)
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = tc::wait(&empty[st], ph, abort_flag, p.status, kWaitNs))) break;
          mbar_arrive_expect_tx(&full[st], C::B_BYTES);
          tc::tma_load_2d(b_base + st * C::B_BYTES, &p.tm_x, &full[st], kb * kBlk, t.row0);
          if (++st == C::STAGES) st = 0, ph ^= 1;
        }
    }
  } else if (warp == kSWarpMma) {
    grid_dependency_wait();
    if (lane == 0) {
      constexpr uint32_t idesc = tc::idesc_f16_f32(128, NT);
      const uint64_t ad0 = tc::sdesc_sw128(smem_addr(a_base)), bd0 = tc::sdesc_sw128(smem_addr(b_base));
      int st = 0, ph = 0, ac = 0, aph = 1, e = 0;
      bool ok = true;
      Tile t;
      for (int it = first; ok && it < p.items && decode(p, it, NT, kBlk, starts, t, e); it += step)
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = tc::wait(&acc_empty[ac], aph, abort_flag, p.status, kWaitNs))) break;
          if (!(ok = tc::wait(&full[st], ph, abort_flag, p.status, kWaitNs, 200))) break;
          tc::fence_after_sync();
          mma_block(tmem + ac * NT, ad0 + static_cast<uint64_t>((st * C::A_BYTES) >> 4),
                    bd0 + static_cast<uint64_t>((st * C::B_BYTES) >> 4), idesc);
          tc::commit(&empty[st]);
          tc::commit(&acc_full[ac]);
          if (++st == C::STAGES) st = 0, ph ^= 1;
          if (++ac == C::ACCS) ac = 0, aph ^= 1;
        }
    }
    __syncwarp();
  } else if (warp == kSWarpScale) {
    // sx * sw of four blocks and NT tokens per slot; lane l takes block l % 4 of rows
    // l / 4 + 8 j
    grid_dependency_wait();
    int sl = 0, ph = 1, e = 0;
    bool ok = true;
    Tile t;
    for (int it = first; ok && it < p.items && decode(p, it, NT, kBlk, starts, t, e); it += step) {
      const int i = lane & 3, r0 = lane >> 2;
      const float* sw = p.w_scale + (static_cast<size_t>(t.expert) * p.NB + t.n0 / kBlk) * p.KB + i;
      const float* sx = p.x_scale + static_cast<size_t>(t.row0 + r0) * p.KB + i;
      const int valid = t.row_end - t.row0 - r0;
      for (int kb = kb0; kb < kb1; kb += 4) {
        const bool in = kb + i < kb1;
        const float w = in ? sw[kb] : 0.f;
        float x[NT / 8];
#pragma unroll
        for (int j = 0; j < NT / 8; ++j) x[j] = in && 8 * j < valid ? sx[static_cast<size_t>(8 * j) * p.KB + kb] : 0.f;
        if (!(ok = wait_warp(&sc_empty[sl], ph, abort_flag, p.status))) break;
        float* sc = sc_base + (sl * 4 + i) * C::SC_ROW + r0;
#pragma unroll
        for (int j = 0; j < NT / 8; ++j) sc[8 * j] = x[j] * w;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[sl]);
        if (++sl == C::SC_SLOTS) sl = 0, ph ^= 1;
      }
    }
  } else {
    grid_dependency_wait();   // the kernels before may still use y
    int ac = 0, aph = 0, sl = 0, sph = 0, e = 0;
    bool ok = true;
    Tile t;
    for (int it = first; ok && it < p.items && decode(p, it, NT, kBlk, starts, t, e); it += step) {
      float T[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) T[j] = 0.f;
      for (int kb = kb0; kb < kb1; ++kb) {
        const int i = (kb - kb0) & (C::SC_PER - 1);
        if (i == 0 && !(ok = wait_warp(&sc_full[sl], sph, abort_flag, p.status))) break;
        if (!(ok = wait_warp(&acc_full[ac], aph, abort_flag, p.status))) break;
        tc::fence_after_sync();
        const uint32_t ta = tmem + (static_cast<uint32_t>(32 * warp) << 16) + ac * NT;
        const float* sc = sc_base + (sl * C::SC_PER + i) * C::SC_ROW;
        // 16 columns are multiplied while the next 16 load
        uint32_t v[2][16];
        tc::tmem_ld16_async(ta, v[0]);
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          uint32_t (&now)[16] = v[(c >> 4) & 1];
          tc::tmem_wait_ld(now);
          if (c + 16 < NT) tc::tmem_ld16_async(ta + c + 16, v[((c >> 4) & 1) ^ 1]);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(sc + c + j);
            fma2v(T[c + j], T[c + j + 1], f.x, f.y, __uint_as_float(now[j]), __uint_as_float(now[j + 1]));
            fma2v(T[c + j + 2], T[c + j + 3], f.z, f.w, __uint_as_float(now[j + 2]), __uint_as_float(now[j + 3]));
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&acc_empty[ac]);
          if (i == C::SC_PER - 1 || kb == kb1 - 1) mbar_arrive(&sc_empty[sl]);
        }
        if (++ac == C::ACCS) ac = 0, aph ^= 1;
        if (i == C::SC_PER - 1 || kb == kb1 - 1) {
          if (++sl == C::SC_SLOTS) sl = 0, sph ^= 1;
        }
      }
      if (!ok) break;
      const int o = 32 * warp + lane, n = t.n0 + o;
      const int valid = t.row_end - t.row0;
      if (p.split > 1) {
        // every copy has landed and every MMA is done: the ring is free
        float* mine = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (j < valid) mine[j * kBlk + o] = T[j];
      } else if (n < p.N) {
        const float bs = p.bias != nullptr ? __uint_as_float(static_cast<uint32_t>(p.bias[n]) << 16) : 0.f;
        uint16_t* yp = p.y + static_cast<size_t>(t.row0) * p.N + n;
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (j < valid) yp[static_cast<size_t>(j) * p.N] = static_cast<uint16_t>(f32_to_bf16_bits(T[j] + bs));
      }
    }
  }
  __syncwarp();

  if (p.split > 1) {
    // One item per cluster: CTA r adds the parts of tokens r, r + split, ... in the
    // order of the parts. A warp takes a token, 4 outputs a lane, with the loads of
    // all parts in flight at once.
    cluster_arrive();
    cluster_wait();
    int e = 0;
    Tile t;
    if (decode(p, first, NT, kBlk, starts, t, e) && !*abort_flag) {
      const int n = t.n0 + 4 * lane;
      if (n < p.N) {
        float b[4] = {0.f, 0.f, 0.f, 0.f};
        if (p.bias != nullptr) {
          const uint2 bb = *reinterpret_cast<const uint2*>(p.bias + n);
          b[0] = bf16_lo(bb.x), b[1] = bf16_hi(bb.x), b[2] = bf16_lo(bb.y), b[3] = bf16_hi(bb.y);
        }
        for (int j = part + warp * p.split; j < t.row_end - t.row0; j += C::THREADS / 32 * p.split) {
          const uint32_t at = smem_addr(smem) + (j * kBlk + 4 * lane) * 4;
          float4 v[kMaxSplit];
#pragma unroll
          for (int r = 0; r < kMaxSplit; ++r)
            if (r < p.split) v[r] = ld_cluster_f32x4(at, r);
          float4 s = v[0];
#pragma unroll
          for (int r = 1; r < kMaxSplit; ++r)
            if (r < p.split) s.x += v[r].x, s.y += v[r].y, s.z += v[r].z, s.w += v[r].w;
          *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(t.row0 + j) * p.N + n) =
              make_uint2(pack_bf16x2(s.x + b[0], s.y + b[1]), pack_bf16x2(s.z + b[2], s.w + b[3]));
        }
      }
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }

  if (*abort_flag) {   // let copies and MMAs in flight land before the shared memory goes away
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kSWarpMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// tile form
// ---------------------------------------------------------------------------

constexpr int TM = 128, TN = 256;             // rows and outputs of a tile
constexpr int T_A = TM * 128, T_B = TN * 128;
constexpr int T_STAGES = 4;
constexpr int T_ACCS = 2;                      // accumulators of 256 columns: all 512 of tensor memory
constexpr int T_SC_SLOTS = 3;                  // scale slots of 4 blocks x 2 output halves x 128 rows
constexpr int T_SC_ROW = 2 * TM + 8;           // 8 rows x 4 blocks of a slot lie in 32 banks
constexpr int T_SC_FLOATS = 4 * T_SC_ROW;
constexpr int T_SC = T_SC_SLOTS * T_SC_FLOATS * 4;
constexpr int T_OUT = 8 * 32 * 64;             // per epilogue warp, 64 bytes of its 32 rows on their way out
constexpr int T_SMEM = T_STAGES * (T_A + T_B) + T_SC + T_OUT + 512 + (kMaxExperts + 1 + 12 + 3) / 4 * 16 + 1024;
static_assert(T_SMEM <= 232448, "shared memory per CTA");
// Blocks go in groups of four: block i of a group has stage i and accumulator i % 2,
// so that the loops over a group know their barriers, and its scales are one slot. A
// work item's last group is filled up with blocks that only pass the barriers
// (counters in place of groups: 4096 x 11008 x 4096 171 us against 163). Every waiter
// meets every phase of the barriers that it waits on.
static_assert(T_STAGES == 4 && T_ACCS == 2, "a group of four blocks");
// Warps 0-7 epilogue (warp w: TMEM lanes 32 (w % 4), outputs 128 (w / 4) ..),
// 8 copies, 9 scales, 10 and 11 MMA issuers of the even and odd blocks: a
// thread's MMAs queue behind its own commits, so with two issuers one
// accumulates while the other's block completes.
constexpr int kTEpi = 8, kTWarpLoad = 8, kTWarpScale = 9, kTWarpMma = 10;
constexpr int kTThreads = 384;

struct Work {
  Tile t;
  int kb0, kb1;
  int part;   // index of its part sums, or -1
};
W4_DEV bool decode_work(const Params& p, int it, const int32_t* starts, Work& w, int& e) {
  w.kb0 = 0;
  w.kb1 = p.KB;
  w.part = -1;
  if (it >= p.full) {
    const int j = it - p.full, tile = j / p.parts, part = j - tile * p.parts;
    w.kb0 = part_start(p.KB, part, p.parts);
    w.kb1 = part_start(p.KB, part + 1, p.parts);
    w.part = j;
    it = p.full + tile;
  }
  return decode(p, it, TM, TN, starts, w.t, e);
}

__global__ void __launch_bounds__(kTThreads, 1) tile_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* a_base = smem;
  uint8_t* b_base = a_base + T_STAGES * T_A;
  float* sc_base = reinterpret_cast<float*>(b_base + T_STAGES * T_B);
  uint4* out_base = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(sc_base) + T_SC);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(out_base) + T_OUT);
  uint64_t* done = full + T_STAGES;        // a block's MMAs: its stage is free and its accumulator complete
  uint64_t* acc_empty = done + T_STAGES;
  uint64_t* sc_full = acc_empty + T_ACCS;
  uint64_t* sc_empty = sc_full + T_SC_SLOTS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sc_empty + T_SC_SLOTS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int32_t* starts = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(full) + 512);
  int32_t* warp_sum = starts + kMaxExperts + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < T_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&done[i], 1);
    }
    for (int i = 0; i < T_ACCS; ++i) mbar_init(&acc_empty[i], kTEpi);
    for (int i = 0; i < T_SC_SLOTS; ++i) {
      mbar_init(&sc_full[i], 1);
      mbar_init(&sc_empty[i], kTEpi);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTWarpMma) tc::tmem_alloc(tmem_holder, T_ACCS * TN);
  if (warp == kTWarpLoad && lane == 0) {
    tc::prefetch_tmap(&p.tm_x);
    tc::prefetch_tmap(&p.tm_w);
  }
  if (p.offsets != nullptr) {
    if (!p.offsets_ready) grid_dependency_wait();   // the routing may be running still
    tile_starts<kTThreads>(p, TM, starts, warp_sum);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  launch_dependents();
  const uint32_t tmem = *tmem_holder;
  const int KB = p.KB;

  if (warp >= kTEpi) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kTWarpLoad) {
      int st = 0, ph = 1, e = 0;
      bool ok = true, waited = false;
      Work w;
      for (long long it = blockIdx.x; ok && it < p.items && decode_work(p, it, starts, w, e); it += gridDim.x)
        for (int kb = w.kb0; kb < w.kb1 || st != 0; ++kb) {
          if (!(ok = wait_warp(&done[st], ph, abort_flag, p.status))) break;
          if (kb >= w.kb1) {
            if (elect_one()) mbar_arrive(&full[st]);   // a filler
          } else {
            if (elect_one()) {
              mbar_arrive_expect_tx(&full[st], T_A + T_B);
              tc::tma_load_3d(b_base + st * T_B, &p.tm_w, &full[st], kb * kBlk, w.t.n0, w.t.expert);
            }
            if (!waited) grid_dependency_wait();   // the codes come from the kernel before
            waited = true;
            if (elect_one()) tc::tma_load_2d(a_base + st * T_A, &p.tm_x, &full[st], kb * kBlk, w.t.row0);
          }
          if (++st == T_STAGES) st = 0, ph ^= 1;
        }
    } else if (warp == kTWarpScale) {
      // sx * sw of four blocks, both output halves and the tile's 128 rows per slot. Lane
      // l takes block l % 4 of rows l / 4 + 8 j, so that a load reads 8 rows' 16 bytes
      // (with a lane to a row, 32 sectors: 4096 x 11008 x 4096 177 us against 171).
      grid_dependency_wait();
      int sl = 0, ph = 1, e = 0;
      bool ok = true;
      Work w;
      for (long long it = blockIdx.x; ok && it < p.items && decode_work(p, it, starts, w, e); it += gridDim.x) {
        const Tile& t = w.t;
        const int nb = t.n0 / kBlk;
        const int i = lane & 3, r0 = lane >> 2;
        const float* sw0 = p.w_scale + (static_cast<size_t>(t.expert) * p.NB + nb) * KB + i;
        const float* sw1 = nb + 1 < p.NB ? sw0 + KB : sw0;
        const float* sx = p.x_scale + static_cast<size_t>(t.row0 + r0) * KB + i;
        const int valid = t.row_end - t.row0 - r0;
        for (int kb = w.kb0; kb < w.kb1; kb += 4) {
          const bool in = kb + i < w.kb1;
          const float w0 = in ? sw0[kb] : 0.f, w1 = in ? sw1[kb] : 0.f;
          float x[16];
          const float* at = sx + kb;
          int down = 8 * KB;
          asm volatile("" : "+r"(down));   // 16 addresses kept over the loop would not fit the registers
#pragma unroll
          for (int j = 0; j < 16; ++j, at += down) x[j] = in && 8 * j < valid ? *at : 0.f;
          if (!(ok = wait_warp(&sc_empty[sl], ph, abort_flag, p.status))) break;
          float* sc = sc_base + sl * T_SC_FLOATS + i * T_SC_ROW + r0;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            sc[8 * j] = x[j] * w0;
            sc[TM + 8 * j] = x[j] * w1;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[sl]);
          if (++sl == T_SC_SLOTS) sl = 0, ph ^= 1;
        }
      }
    } else {
      grid_dependency_wait();
      const bool leader = elect_one();
      const int mine = warp - kTWarpMma;   // blocks and accumulator of this parity
      constexpr uint32_t idesc = tc::idesc_f16_f32(TM, TN);
      const uint64_t ad0 = tc::sdesc_sw128(smem_addr(a_base)), bd0 = tc::sdesc_sw128(smem_addr(b_base));
      int ph = 0, e = 0;
      bool ok = true;
      Work w;
      for (long long it = blockIdx.x; ok && it < p.items && decode_work(p, it, starts, w, e); it += gridDim.x)
        for (int kb = w.kb0 + mine; ok && kb < w.kb1 + mine; kb += 4) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int st = 2 * j + mine;
            // the operands are there long before: the accumulator, waited for last, is what holds the MMAs up
            if (!(ok = wait_warp(&full[st], ph, abort_flag, p.status))) break;
            if (!(ok = wait_warp(&acc_empty[mine], j ^ 1, abort_flag, p.status))) break;
            tc::fence_after_sync();
            if (leader) {
              if (kb + 2 * j < w.kb1)
                mma_block(tmem + mine * TN, ad0 + static_cast<uint64_t>((st * T_A) >> 4), bd0 + static_cast<uint64_t>((st * T_B) >> 4), idesc);
              tc::commit(&done[st]);
            }
            __syncwarp();
          }
          ph ^= 1;
        }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // y and the part sums may still be in use by the kernels before: stores wait for
    // them here, not only through the copies of the codes
    grid_dependency_wait();
    const int q = warp & 3, half = warp >> 2;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * q) << 16) + 128 * half;
    const float* sc_mine = sc_base + half * TM + 32 * q + lane;
    int ph = 0, sl = 0, sph = 0, e = 0;
    bool ok = true;
    Work w;
    for (long long it = blockIdx.x; ok && it < p.items && decode_work(p, it, starts, w, e); it += gridDim.x) {
      float T[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) T[j] = 0.f;
      for (int kb = w.kb0; ok && kb < w.kb1; kb += 4) {
        if (!(ok = wait_warp(&sc_full[sl], sph, abort_flag, p.status))) break;
        const float* sc_now = sc_mine + sl * T_SC_FLOATS;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = sc_now[i * T_SC_ROW];
          if (!(ok = wait_warp(&done[i], ph, abort_flag, p.status))) break;
          tc::fence_after_sync();
          if (kb + i >= w.kb1) {
            if (lane == 0) mbar_arrive(&acc_empty[i & 1]);   // a filler
            continue;
          }
          const uint32_t ta = t_lane + (i & 1) * TN;
          // 16 columns are multiplied while the next 16 load
          uint32_t v[2][16];
          tc::tmem_ld16_async(ta, v[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            tc::tmem_wait_ld(v[c & 1]);
            if (c < 7) {
              tc::tmem_ld16_async(ta + 16 * (c + 1), v[(c + 1) & 1]);
            } else {
              tc::fence_before_sync();
              __syncwarp();
              if (lane == 0) mbar_arrive(&acc_empty[i & 1]);   // the accumulator is in registers
            }
#pragma unroll
            for (int j = 0; j < 16; j += 2)
              fma2(T[16 * c + j], T[16 * c + j + 1], f, __uint_as_float(v[c & 1][j]), __uint_as_float(v[c & 1][j + 1]));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_empty[sl]);
        ph ^= 1;
        if (++sl == T_SC_SLOTS) sl = 0, sph ^= 1;
      }
      if (!ok) break;
      const int row0 = w.t.row0 + 32 * q, n0 = w.t.n0 + 128 * half, row_end = w.t.row_end;
      uint4* buf = out_base + warp * 128;
      if (w.part >= 0) {
        float* ps = p.part_sums + (static_cast<size_t>(w.part) * TM + 32 * q) * TN + 128 * half;
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 16) {
          uint4 v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            v[c] = make_uint4(__float_as_uint(T[c0 + 4 * c]), __float_as_uint(T[c0 + 4 * c + 1]),
                              __float_as_uint(T[c0 + 4 * c + 2]), __float_as_uint(T[c0 + 4 * c + 3]));
          rows_out(buf, v, [&](int r, int c, const uint4& x) {
            if (row0 + r < row_end) *reinterpret_cast<uint4*>(ps + static_cast<size_t>(r) * TN + c0 + 4 * c) = x;
          });
        }
      } else {
        uint16_t* yp = p.y + static_cast<size_t>(row0) * p.N + n0;
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          if (n0 + c0 >= p.N) break;
          uint4 v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float* x = T + c0 + 8 * c;
            float b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (p.bias != nullptr && n0 + c0 + 8 * c < p.N) {
              const uint4 bb = *reinterpret_cast<const uint4*>(p.bias + n0 + c0 + 8 * c);
              b[0] = bf16_lo(bb.x), b[1] = bf16_hi(bb.x), b[2] = bf16_lo(bb.y), b[3] = bf16_hi(bb.y);
              b[4] = bf16_lo(bb.z), b[5] = bf16_hi(bb.z), b[6] = bf16_lo(bb.w), b[7] = bf16_hi(bb.w);
            }
            v[c] = make_uint4(pack_bf16x2(x[0] + b[0], x[1] + b[1]), pack_bf16x2(x[2] + b[2], x[3] + b[3]),
                              pack_bf16x2(x[4] + b[4], x[5] + b[5]), pack_bf16x2(x[6] + b[6], x[7] + b[7]));
          }
          rows_out(buf, v, [&](int r, int c, const uint4& x) {
            if (row0 + r < row_end && n0 + c0 + 8 * c < p.N)   // N is a multiple of 8
              *reinterpret_cast<uint4*>(yp + static_cast<size_t>(r) * p.N + c0 + 8 * c) = x;
          });
        }
      }
    }
  }
  __syncwarp();

  if (*abort_flag) {
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kTWarpMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, T_ACCS * TN);
  }
}

// y = bf16(part sums in order + bias) of the tiles that were split.
__global__ void __launch_bounds__(256) join_parts_kernel(const float4* sums, int parts, int tiles,
                                                         int full, int n_tiles, int rows, int N,
                                                         const uint16_t* bias, uint16_t* __restrict__ y) {
  constexpr int kRow = TN / 4;
  launch_dependents();
  grid_dependency_wait();
  const int total = tiles * TM * kRow;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const int tile = i / (TM * kRow), r = i / kRow % TM, c4 = i % kRow;
    const int id = full + tile, row = id / n_tiles * TM + r, n = id % n_tiles * TN + 4 * c4;
    if (row >= rows || n >= N) continue;   // N is a multiple of 8
    const float4* s = sums + (static_cast<size_t>(tile) * parts * TM + r) * kRow + c4;
    float4 a = __ldcg(s);
    for (int j = 1; j < parts; ++j) {
      const float4 b = __ldcg(s + static_cast<size_t>(j) * TM * kRow);
      a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
    }
    if (bias != nullptr) {
      const uint2 b = *reinterpret_cast<const uint2*>(bias + n);
      a.x += bf16_lo(b.x), a.y += bf16_hi(b.x), a.z += bf16_lo(b.y), a.w += bf16_hi(b.y);
    }
    *reinterpret_cast<uint2*>(y + static_cast<size_t>(row) * N + n) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Row tiles of `per` rows that R rows in E segments can need at most.
int64_t row_tiles(const Fp8BlockArgs& a, int per) {
  const int64_t whole = (a.R + per - 1) / per;
  return a.expert_offsets == nullptr ? whole : (a.R < whole + a.E ? a.R : whole + a.E);
}

// Clusters of n CTAs, one an SM, that the device holds at once: they do not cross a
// group of SMs, so that this is less than the SMs divided by n. Asked once per device
// and n (any stream kernel would do: the answer counts one CTA an SM for all of them).
int one_cta_clusters(int n) {
  using C = Stream<128, false>;
  static std::atomic<int> known[64][kMaxSplit + 1];   // answer + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
  int v = known[dev][n].load(std::memory_order_relaxed);
  if (v == 0) {
    PdlLaunch pl(static_cast<unsigned>(n), C::THREADS, C::SMEM, nullptr, n);
    if (cudaFuncSetAttribute(stream_kernel<128, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&v, stream_kernel<128, false>, &pl.cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    known[dev][n].store(++v, std::memory_order_relaxed);
  }
  return v - 1;
}
}  // namespace

// The same for `ctas` (1 or 2) an SM: with two, a group of S SMs holds 2S / n clusters
// of n, at least as many as S / ceil(n / 2) and as twice S / n.
int clusters_held(int n, int ctas) {
  const int one = one_cta_clusters(n);
  if (ctas == 1) return one;
  const int half = n > 2 ? one_cta_clusters((n + 1) / 2) : 0;
  return half > 2 * one ? half : 2 * one;
}

namespace {

template <int NT, bool kQuant>
cudaError_t run_stream(const Fp8BlockArgs& a, Params& p, cudaStream_t s) {
  using C = Stream<NT, kQuant>;
  cudaError_t e = kQuant ? cudaSuccess : encode(&p.tm_x, a.qx, a.K, a.R, 0, NT);
  if (e != cudaSuccess) return e;
  e = encode(&p.tm_w, a.qweight, a.K, a.N, a.E, kBlk);
  if (e != cudaSuccess) return e;
  p.n_tiles = static_cast<int>((a.N + kBlk - 1) / kBlk);
  const int64_t items = row_tiles(a, NT) * p.n_tiles;
  if (items > kMaxItems) return cudaErrorInvalidConfiguration;
  p.items = static_cast<int>(items);
  const int64_t slots = static_cast<int64_t>(current_sm_count()) * C::CTAS;
  // The largest cluster that leaves every part 2.5 blocks on average and all clusters
  // resident at once: 16 x 4096 x 4096 takes 11.1 us in clusters of 2 and 8.0 of 8; 16 x
  // 6144 x 4096 (48 items) 9.2 in clusters of 5, while 48 of 6 take two rounds and 15.9.
  p.split = 1;
  if (a.expert_offsets == nullptr)
    for (int n = kMaxSplit; n > 1 && p.split == 1; --n)
      if (2 * p.KB >= 5 * n && items <= clusters_held(n, C::CTAS)) p.split = n;
  const int64_t grid = p.split > 1 ? items * p.split : (items < slots ? items : slots);
  return start<stream_kernel<NT, kQuant>>(p, grid, C::THREADS, C::SMEM, p.split, s);
}

}  // namespace

// The dense tile form's work: whole waves of whole tiles, and the r tiles of a
// last, partly filled wave cut along k into as many parts as fit the SMs at once.
// That takes KB - KB / s blocks of 0.48 us off the last wave and costs about
// kSplitBlocks of them: the sums of 128 KB a part, written and read back, and the
// join's launch. Measured whole / split: 517 x 11008 x 4096 (r = 63, two parts) 37.2
// / 34.4 us, 300 x 2048 x 14336 (24, six) 52.2 / 22.6, 700 x 14336 x 8192 (32, four)
// 99 / 84. More parts than SMs lose: 256 x 11008 x 4096 (86, three) 22.1 / 31.8.
// The SM count is a GB300's whatever the device, so that the workspace is the same
// everywhere.
constexpr int kPlanSms = 152, kSplitBlocks = 12;
struct Plan {
  int64_t full, tail;
  int parts;
};
static Plan tile_plan(int64_t R, int64_t N, int64_t K) {
  const int64_t tiles = ((R + TM - 1) / TM) * ((N + TN - 1) / TN), r = tiles % kPlanSms, KB = (K + kBlk - 1) / kBlk;
  if (r == 0) return {tiles, 0, 1};
  int64_t s = kPlanSms / r;
  if (s > 16) s = 16;
  if (s > KB) s = KB;   // every part has a block
  if (s < 2 || (KB + s - 1) / s + kSplitBlocks >= KB) return {tiles, 0, 1};
  return {tiles - r, r, static_cast<int>(s)};
}

// The tile form is for more rows per weight tile than the stream form takes at
// once. Experts: above 56 rows an expert on average, where the stream form would have
// to read many weight tiles twice (64 experts of 2816 x 2048, stream / tile: 48 rows
// 69.9 / 72.5 us, 56 rows 73.0 / 73.0, 64 rows 81 / 74, 96 rows 106 / 79). Dense:
// above 128 rows (4096 x 4096 at 129 rows 18.2 / 15.4 us, 11008 x 4096 41 / 21), or above
// 64 where the N tiles alone fill more than half of the SMs, so that no cluster
// shares their k (96 rows, stream / tile: 11008 x 4096 22.2 / 20.1, 131072 x 2048
// 70 / 55, but 4096 x 4096 12.1 / 15.3 and 2048 x 8192 13.8 / 17.3).
static bool tile_form(int64_t R, int64_t N, int64_t E, bool experts) {
  if (experts) return R > 56 * E;
  return R > 128 || (R > 64 && 2 * ((N + kBlk - 1) / kBlk) > kPlanSms);
}

bool fp8_block_fuses(int64_t R, bool experts) { return !experts && R <= kFuseRows; }

size_t fp8_block_part_bytes(int64_t R, int64_t N, int64_t K) {
  if (!tile_form(R, N, 1, false)) return 0;
  const Plan p = tile_plan(R, N, K);
  return p.parts > 1 ? static_cast<size_t>(p.tail) * p.parts * TM * TN * sizeof(float) : 0;
}

cudaError_t launch_fp8_block(const Fp8BlockArgs& a, cudaStream_t s) {
  Params p;
  memset(&p, 0, sizeof(p));
  p.x_scale = a.x_scale;
  p.w_scale = a.w_scale;
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.y = static_cast<uint16_t*>(a.y);
  p.offsets = a.expert_offsets;
  p.offsets_ready = a.offsets_ready;
  p.E = a.E;
  p.rows = static_cast<int>(a.R);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.KB = static_cast<int>((a.K + kBlk - 1) / kBlk);
  p.NB = static_cast<int>((a.N + kBlk - 1) / kBlk);
  p.split = 1;
  p.status = a.status;
  p.x = static_cast<const uint4*>(a.x);
  p.x_f16 = a.x_f16;
  const bool experts = a.expert_offsets != nullptr;
  if (!tile_form(a.R, a.N, a.E, experts)) {
    // The smallest token tile that holds a call's rows, or an expert's on average: at
    // 11008 x 4096 20 rows take 17.5 us in tiles of 16 and 12.1 in one of 32, 48
    // rows 18.0 in tiles of 32 and 14.2 in one of 64, while 16 rows take 11.6 and 11.9,
    // 33 rows 13.8 and (in one of 128) 21; 64 experts of 2816 x 2048 with 12 rows 63.5 in
    // tiles of 16 and 64.6 of 32, with 20 rows 69.7 and 65.1, with 40 rows 77.7
    // in tiles of 32 and 70.2 of 64.
    const int64_t rows = (a.R + a.E - 1) / a.E;
    if (rows <= 16) return a.x != nullptr ? run_stream<16, true>(a, p, s) : run_stream<16, false>(a, p, s);
    if (rows <= 32) return run_stream<32, false>(a, p, s);
    // Above 40 dense rows two tiles of 32, where clusters of 4 have room for them and the
    // weights, read twice, are few: the join of wide tiles costs more. 64 x 4096 x 4096
    // 10.1 us against 11.4, 64 x 2048 x 8192 11.0 / 12.2, 40 x 4096 x 4096 10.1 / 9.7, 64 x
    // 6144 x 4096 (no room) 12.9 / 12.0, 64 x 4096 x 14336 (59 MB) 20.5 / 18.7.
    const bool twice = !experts && rows > 40 && 2 * ((a.N + kBlk - 1) / kBlk) <= clusters_held(4, Stream<32, false>::CTAS) &&
                       a.N * a.K <= int64_t{1} << 25;
    if (rows <= 64) return twice ? run_stream<32, false>(a, p, s) : run_stream<64, false>(a, p, s);
    return run_stream<128, false>(a, p, s);
  }
  cudaError_t e = encode(&p.tm_x, a.qx, a.K, a.R, 0, TM);
  if (e != cudaSuccess) return e;
  e = encode(&p.tm_w, a.qweight, a.K, a.N, a.E, TN);
  if (e != cudaSuccess) return e;
  p.n_tiles = static_cast<int>((a.N + TN - 1) / TN);
  const int64_t items = row_tiles(a, TM) * p.n_tiles;
  if (items > kMaxItems) return cudaErrorInvalidConfiguration;
  p.items = p.full = static_cast<int>(items);
  p.parts = 1;
  const Plan plan = experts ? Plan{0, 0, 1} : tile_plan(a.R, a.N, a.K);
  if (plan.parts > 1 && a.part_bytes >= fp8_block_part_bytes(a.R, a.N, a.K)) {
    p.full = static_cast<int>(plan.full);
    p.parts = plan.parts;
    p.part_sums = a.part_sums;
    p.items = static_cast<int>(plan.full + plan.tail * plan.parts);
  }
  const int64_t sms = current_sm_count();
  e = start<tile_kernel>(p, p.items < sms ? p.items : sms, kTThreads, T_SMEM, 1, s);
  if (e != cudaSuccess || p.parts == 1) return e;
  const int64_t want = plan.tail * TM * (TN / 4) / 256, most = sms * 8;
  PdlLaunch pl(static_cast<unsigned>(want < most ? want : most), 256, 0, s);
  return cudaLaunchKernelEx(&pl.cfg, join_parts_kernel, reinterpret_cast<const float4*>(p.part_sums), p.parts,
                            static_cast<int>(plan.tail), p.full, p.n_tiles, p.rows, p.N, p.bias, p.y);
}

}  // namespace w4
