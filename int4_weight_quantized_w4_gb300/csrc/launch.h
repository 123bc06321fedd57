// Internal host-side launch functions, one per kernel family. The public
// entry points in api.cu validate arguments and then call these; each returns
// the cudaError_t of its launch.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "w4.h"

namespace w4 {

// SMs of the current device, asked on every call: the runtime answers from its
// own cache, the status is checked before the value is used, and the answer
// is right for whichever device the caller has made current.
inline int current_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      n <= 0)
    n = 152;
  return n;
}

// Polls a bounded wait makes before it gives up (about a second of spinning).
constexpr long long kWaitLimit = 1LL << 24;

// A launch that may start while the kernel before it on the stream finishes
// (programmatic dependent launch): the kernel waits for it (griddepcontrol.wait)
// before it reads anything that kernel writes or writes anything it reads. With
// `cluster` > 1, in clusters of that many blocks.
struct PdlLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  PdlLaunch(unsigned grid, unsigned block, size_t smem, cudaStream_t s, unsigned cluster = 1) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
  }
  PdlLaunch(const PdlLaunch&) = delete;
  PdlLaunch& operator=(const PdlLaunch&) = delete;
};

// status: the device status word (a timed-out wait records W4_ERR_TIMEOUT there).
cudaError_t launch_quant_per_token(const void* x, bool x_f16, int64_t M, int64_t K, bool fp8, void* q,
                                   float* scale, unsigned int* status, cudaStream_t s);

struct W4A16Args {
  const void* x;
  const void* qweight;
  const void* w_scale;
  bool scale_bf16;
  const void* zeros;
  const void* bias;
  void* y;
  int64_t M, N, K;
  int32_t group;  // effective group (K when the caller passed -1)
  unsigned int* status;
  // host entry point, page-locked host buffers (device addresses): x is copied
  // from x_host into x by the L2-prefetch grid, y written to y_host as well
  const void* x_host = nullptr;
  void* y_host = nullptr;
};
cudaError_t launch_w4a16(const W4A16Args& a, cudaStream_t s);
// Per-token quantization whose output is the codes' exact fp16 values in the
// W4A8 operand order (fp16 [M, K] into `wide`), plus the fp32 scales.
cudaError_t launch_quant_widen(const void* x, int64_t M, int64_t K, bool fp8, void* wide, float* scale,
                               unsigned int* status, cudaStream_t s);
// Shared memory the decode kernel needs for one token row beside a minimal ring.
size_t w4a16_smem_bytes(int64_t N, int64_t K, int32_t group);

struct W4A8Args {
  const void* act;        // int8 [M,K] (dense) or e4m3 [R,K] (experts)
  const float* x_scale;   // [M] (ignored for partials)
  const void* qweight;    // GPTQ [K/8,N] (dense) or CT [E,N,K/8] (experts)
  const void* w_scale;    // fp16 [G,N] (dense) or [E,N,G] (experts)
  const void* bias;       // bf16 [N] or nullptr
  void* out;              // bf16 [M,N], or int32 [M,G,N] for partials
  const int32_t* expert_offsets;  // device [E+1] (experts only)
  int32_t E;
  int64_t M, N, K;
  int32_t group;          // effective group
  bool partials;          // write int32 group partials instead of y
  unsigned int* status;
  void* workspace;        // fp16 [rows, K]: the activations widened once per call
  bool prewidened;        // the workspace already holds them (act unused)
  bool fp8_act;           // experts: act holds e4m3 codes [R, K] that the fp8 tensor path reads directly
  size_t workspace_bytes; // dense y: a workspace this large may also hold split-K partial sums
};
size_t w4a8_workspace_bytes(int64_t rows, int64_t K);
// The dense W4A8 workspace with room for the split-K partial sums that
// M x N x K at this group would use (fp32 [splits][M][N] after the widened
// activations); equal to w4a8_workspace_bytes when the GEMM is not split.
size_t w4a8_workspace_bytes_split(int64_t M, int64_t N, int64_t K, int32_t group);
// Sets the calling thread's w4_last_error() message and returns `st`.
w4_status report_error(w4_status st, const char* msg);
cudaError_t launch_w4a8_dense(const W4A8Args& a, cudaStream_t s);
cudaError_t launch_w4afp8_experts(const W4A8Args& a, cudaStream_t s);
// Expert GEMMs whose (effective) group is a multiple of 32 run on the fp8
// tensor path (kind::f8f6f4, 32 k per MMA); others widen to fp16 first.
bool w4afp8_fp8_path(int32_t group);

cudaError_t launch_quantize_groupwise(const void* w, bool f16, int64_t N, int64_t K, int32_t group, uint8_t* packed,
                                      float* scale, float* zero, cudaStream_t s);
cudaError_t launch_xor88(const void* src, void* dst, int64_t n_bytes, cudaStream_t s);
cudaError_t launch_embedding_gather(const int32_t* ids, int64_t T, const void* table, const float* scale,
                                    const float* zero, int64_t V, int64_t D, int32_t group, void* out,
                                    unsigned int* status, cudaStream_t s);
cudaError_t launch_lm_head(const void* h, int64_t M, const void* table, const float* scale, const float* zero,
                           int64_t V, int64_t D, int32_t group, void* y, cudaStream_t s);
cudaError_t launch_quant_gather(const void* x, int64_t T, int64_t K, const int32_t* rows, int64_t R, bool fp8,
                                bool widen, void* q, float* scale, unsigned int* status, cudaStream_t s);
size_t moe_route_workspace_bytes(int64_t T, int32_t E);
cudaError_t launch_moe_route(const void* logits, bool bf16, int64_t T, int32_t E, int32_t k, bool renorm,
                             int32_t* ids, float* wts, int32_t* offsets, int32_t* row_token, int32_t* row_of,
                             void* workspace, cudaStream_t s);
struct MoeRouteArgs {
  const void* logits;      // [T, E], bf16 or fp32
  const float* bias;       // [E] or null
  int64_t T;
  int32_t E, k, n_group, topk_group;
  bool bf16, softmax, renorm;
  float factor;
  int32_t* ids;            // outputs as w4_moe_route
  float* wts;
  int32_t *offsets, *row_token, *row_of;
  void* workspace;
};
size_t moe_route_grouped_workspace_bytes(int64_t T, int32_t E);
cudaError_t launch_moe_route_grouped(const MoeRouteArgs& a, cudaStream_t s);
cudaError_t launch_silu_mul_quant(const void* h, int64_t R, int64_t I, void* q, float* scale, void* act,
                                  cudaStream_t s);
cudaError_t launch_moe_combine(const void* y, int64_t R, int64_t H, const float* w, const int32_t* row_of, int64_t T,
                               int32_t k, void* out, unsigned int* status, cudaStream_t s);
// e4m3 codes and fp32 scales per row and 128 columns of x [*, K] (bf16, or fp16), or of silu(gate) * up of x
// [*, 2K] (silu, bf16); gather (may be null): source row of each of the M output rows, checked against T. late: a
// programmatic dependent starts only when every kernel before this one is done.
// M rows of K fit one grid (quant_block_fits).
cudaError_t launch_quant_block(const void* x, bool f16, bool silu, int64_t M, int64_t K, const int32_t* gather,
                               int64_t T, bool late, void* q, float* scale, unsigned int* status, cudaStream_t s);
bool quant_block_fits(int64_t M, int64_t K);
// Rows gather[r] of quantized (src, src_scale) [T, K], which the kernel launched just before writes, as row r of (dst, dst_scale);
// late, as above.
cudaError_t launch_gather_block_rows(const void* src, const float* src_scale, int64_t T, int64_t K,
                                     const int32_t* gather, int64_t R, void* dst, float* dst_scale,
                                     unsigned int* status, cudaStream_t s);
struct Fp8BlockArgs {
  const void* qx;                 // e4m3 [R, K]
  const float* x_scale;           // [R, ceil(K / 128)]
  const void* qweight;            // e4m3 [E, N, K]
  const float* w_scale;           // [E, ceil(N / 128), ceil(K / 128)]
  const void* bias;               // bf16 [N] or null
  void* y;                        // bf16 [R, N]
  const int32_t* expert_offsets;  // device [E + 1], or null: dense, E = 1
  int32_t E;
  int64_t R, N, K;
  const void* x;                  // where fp8_block_fuses: 16-bit activations [R, K] in place of qx and x_scale
  bool x_f16;
  bool offsets_ready;             // experts: the kernel launched just before lets its dependents go late
  float* part_sums;               // dense: at least fp8_block_part_bytes, 16-byte aligned (or null, 0: the product is not split along K)
  size_t part_bytes;
  unsigned int* status;
};
// fp32 part sums of the dense product's split tiles.
size_t fp8_block_part_bytes(int64_t R, int64_t N, int64_t K);
// Quantized rows of the 16-bit-input forms: codes [R, K], then scales [R, ceil(K / 128)], padded to 16 bytes.
inline size_t fp8_block_workspace_bytes(int64_t R, int64_t K) {
  const size_t n = static_cast<size_t>(R) * static_cast<size_t>(K) + static_cast<size_t>(R) * static_cast<size_t>((K + 127) / 128) * 4;
  return (n + 15) / 16 * 16;
}
// Whether launch_fp8_block takes 16-bit activations.
bool fp8_block_fuses(int64_t R, bool experts);
cudaError_t launch_fp8_block(const Fp8BlockArgs& a, cudaStream_t s);
cudaError_t launch_bounded_wait_selftest(long long limit, unsigned int* status, cudaStream_t s);

}  // namespace w4
