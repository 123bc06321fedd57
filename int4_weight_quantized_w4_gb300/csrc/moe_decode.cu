// The few-token expert layer (moe_decode.cuh) on int4 weights, and what its two units share on
// the host.
#include "moe_decode.cuh"

namespace w4 {
namespace {

template <bool kDown, int kBlocks, bool kWhole>
__global__ void __launch_bounds__(kThreads, 1) moe_decode_int4_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_dyn[];
  Common& c = common_of(smem_dyn);
  prepare(p, c);
  if (kDown) launch_dependents();
  grid_dependency_wait();
  if (!kDown) launch_dependents();
  layer<W4_FMT_INT4, kDown, kBlocks, kWhole>(p, c);
}

// A kernel's code for scales of whole pieces of a warp is shorter: what is not in it need not come from the
// instruction cache (8 tokens 74 us for any group, 70 for these; with more than eight the up kernel would
// spill registers, 109 for 103).
template <bool kDown, bool kWhole>
cudaError_t run_blocks(const MoeDecodeArgs& a, cudaStream_t s) {
  if (a.route.T > 8) return run<moe_decode_int4_kernel<kDown, kDown ? 4 : 2, kDown && kWhole>, W4_FMT_INT4, kDown>(a, s);
  if (kDown && a.route.T > 4) return run<moe_decode_int4_kernel<kDown, kDown ? 2 : 1, kWhole>, W4_FMT_INT4, kDown>(a, s);
  return run<moe_decode_int4_kernel<kDown, 1, kWhole>, W4_FMT_INT4, kDown>(a, s);
}
template <bool kDown>
cudaError_t run_fitting(const MoeDecodeArgs& a, cudaStream_t s) {
  const int steps = (kDown ? a.down_group : a.gate_up_group) / 32;
  if (steps % kPer == 0 && (steps & (steps - 1)) == 0 && (kDown ? a.I : a.H) % (32 * kPer) == 0) return run_blocks<kDown, true>(a, s);
  return run_blocks<kDown, false>(a, s);
}

}  // namespace

bool moe_decode_fits(const MoeDecodeArgs& a) {
  return a.I <= kMaxI && layout_of(a, false).slots >= 2 && layout_of(a, true).slots >= 2;
}

size_t moe_decode_workspace_bytes(int64_t T, int64_t k, int64_t I) {
  return (kMoeChoiceBytes + static_cast<size_t>(T * k) * static_cast<size_t>(4 * I + I / 8) + 15) / 16 * 16;
}

cudaError_t launch_moe_decode(const MoeDecodeArgs& a, cudaStream_t s) {
  if (a.format != W4_FMT_INT4) return launch_moe_decode_fp4(a, s);
  const cudaError_t e = run_fitting<false>(a, s);
  return e == cudaSuccess ? run_fitting<true>(a, s) : e;
}

}  // namespace w4
