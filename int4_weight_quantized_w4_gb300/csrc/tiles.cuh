// What the tensor-core products over segments of rows share: the tiles of a call
// (dense, or of expert segments), cluster and dependent-launch helpers, tensor maps
// and the launch. P is a kernel's parameter struct with offsets, E, rows and n_tiles.
#pragma once

#include <cuda.h>

#include <atomic>
#include <cstring>

#include "common.cuh"
#include "launch.h"
#include "tc.cuh"

namespace w4 {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxSplit = 8;                  // CTAs of a cluster that share a tile's k blocks
// 2 s per wait. A warp that waits for what depends on the kernels before waits for these
// first (griddepcontrol.wait, without a limit), so that their time does not count.
constexpr uint64_t kWaitNs = 2000000000ull;

W4_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
W4_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
W4_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Four floats at shared address `a` of CTA `rank` of the cluster.
W4_DEV float4 ld_cluster_f32x4(uint32_t a, uint32_t rank) {
  float4 v;
  asm volatile("{.reg .b32 t; mapa.shared::cluster.u32 t, %4, %5; ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [t];}"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a), "r"(rank) : "memory");
  return v;
}
// tc::wait by a whole warp with one answer: a warp whose lanes disagreed after a
// time-out would not meet at its next warp-wide instruction.
W4_DEV bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* status) {
  constexpr unsigned kAll = 0xFFFFFFFFu;
  if (__all_sync(kAll, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = tc::globaltimer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i)
      if (__all_sync(kAll, tc::try_wait_suspend(bar, parity, 1000))) return true;
    if (__any_sync(kAll, *abort != 0)) return false;
    if (__any_sync(kAll, tc::globaltimer_ns() - t0 > kWaitNs)) {
      report(status, W4_ERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}
// One lane of a converged warp. Loops that issue copies or MMAs run in the whole
// warp with one lane issuing: descriptors and addresses stay in uniform registers.
W4_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{.reg .pred P; elect.sync _|P, 0xFFFFFFFF; selp.u32 %0, 1, 0, P;}" : "=r"(p));
  return p != 0;
}
W4_DEV void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
W4_DEV void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// First row tile of every expert (tiles of `rows_per` rows), in shared memory:
// starts[e], starts[E] = the total. All threads of the block take part; at
// most kMaxExperts experts. The kernel's seg_bounds(p, e, a, b) gives expert e's rows [a, b).
template <int kThreads, class P>
W4_DEV void tile_starts(const P& p, int rows_per, int32_t* starts, int32_t* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0;
  for (int e0 = 0; e0 < p.E; e0 += kThreads) {
    const int e = e0 + threadIdx.x;
    int n = 0;
    if (e < p.E) {
      int a, b;
      seg_bounds(p, e, a, b);
      n = b > a ? (b - a + rows_per - 1) / rows_per : 0;
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int before = carry, all = carry;
    for (int w = 0; w < kThreads / 32; ++w) {
      const int s = warp_sum[w];
      if (w < warp) before += s;
      all += s;
    }
    if (e < p.E) starts[e] = before + inc - n;
    carry = all;
    __syncthreads();
  }
  if (threadIdx.x == 0) starts[p.E] = carry;
}

struct Tile {
  int n0, row0, row_end, expert;
};
// Item `it` (n tiles fastest) as a tile of `rows_per` rows and `cols_per`
// outputs; false when there are no more. `e` is the caller's cursor over the
// experts: items come in increasing order.
template <class P>
W4_DEV bool decode(const P& p, int it, int rows_per, int cols_per, const int32_t* starts, Tile& t, int& e) {
  const int yt = static_cast<int>(static_cast<unsigned>(it) / static_cast<unsigned>(p.n_tiles));
  t.n0 = (it - yt * p.n_tiles) * cols_per;
  if (p.offsets == nullptr) {
    t.expert = 0;
    t.row0 = yt * rows_per;
    t.row_end = min(t.row0 + rows_per, p.rows);
    return t.row0 < p.rows;
  }
  if (yt >= starts[p.E]) return false;
  while (starts[e + 1] <= yt) ++e;
  int a, b;
  seg_bounds(p, e, a, b);
  t.expert = e;
  t.row0 = a + (yt - starts[e]) * rows_per;
  t.row_end = min(t.row0 + rows_per, b);
  return true;
}

// 64 bytes of every lane's row (four 16-byte chunks) through `buf` (2 KB of this
// warp): put(r, c, v) gets chunk c of row r, four lanes to a row and 8 rows an
// instruction, where the lanes' own stores would touch 32 rows at 16 bytes each.
template <class Put>
W4_DEV void rows_out(uint4* buf, const uint4 (&v)[4], Put put) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 4; ++c) buf[lane * 4 + (c ^ ((lane >> 1) & 3))] = v[c];   // no two of 8 lanes in one bank
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2), c = lane & 3;
    put(r, c, buf[r * 4 + (c ^ ((r >> 1) & 3))]);
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int64_t kMaxItems = int64_t{1} << 30;   // more tiles than any y that fits the device has

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t get_encoder(EncodeTiled* fn) {
  static const EncodeTiled cached = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  if (cached == nullptr) return cudaErrorNotSupported;
  *fn = cached;
  return cudaSuccess;
}

// Rows of K bytes in boxes of box_rows rows x 128 bytes (of box_mats matrices), 128-byte
// swizzle; rows and columns past the tensor arrive as zeros.
// With `plain` bytes given, boxes of that many bytes a row without a swizzle.
cudaError_t encode(CUtensorMap* m, const void* base, int64_t K, int64_t rows, int64_t E, int box_rows, int box_mats = 1,
                   int plain = 0) {
  EncodeTiled fn = nullptr;
  cudaError_t e = get_encoder(&fn);
  if (e != cudaSuccess) return e;
  const cuuint32_t rank = E > 0 ? 3 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)rows, (cuuint64_t)E};
  const cuuint64_t strides[2] = {(cuuint64_t)K, (cuuint64_t)K * (cuuint64_t)rows};
  const cuuint32_t box[3] = {plain > 0 ? (cuuint32_t)plain : 128, (cuuint32_t)box_rows, (cuuint32_t)box_mats}, estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, plain > 0 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Lets a kernel use its dynamic shared memory: once per device, since the call
// costs as much as the rest of the host path put together. A device reset takes
// the setting back; the launch that then fails is repeated with it set again. `most`: the most
// shared memory of any launch, where they differ: a launch that is captured must not fail first.
template <auto kKernel, class P>
cudaError_t start(const P& p, int64_t grid, int threads, int smem, int cluster, cudaStream_t s, int most = 0) {
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  PdlLaunch pl(static_cast<unsigned>(grid), threads, smem, s, cluster);
  if (set.load(std::memory_order_relaxed) & bit) {
    e = cudaLaunchKernelEx(&pl.cfg, kKernel, p);
    if (e != cudaErrorInvalidValue) return e;
    cudaGetLastError();
  }
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most > smem ? most : smem);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&pl.cfg, kKernel, p);
  if (e == cudaSuccess && dev < 64) set.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace
}  // namespace w4
