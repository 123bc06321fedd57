// The few-token expert layer (moe_decode.cuh) on 4-bit floating point weights.
//
// (A form on the block-scaled tensor cores, which multiply the weights as they are, was taken out: it
// needs the activations as 4-bit floats too, sums of several with scales per block. Five terms left 2^-13 of a
// block's largest magnitude, so that a column of 4096 cost the numbers of size 1 beside it 2 %, and nvfp4's
// scales lost all below 2^-17 of a row's. Its times, and this form's: 5 tokens, 96 experts of 1024 x 704 in mxfp4
// 25.6 us, 24.3; 16 tokens, 64 of 2048 x 1408 in nvfp4 104.7, 107 to 115; 8 tokens, 32 of 4096 x 1536 in mxfp4 76, 98.)
#include "moe_decode.cuh"

namespace w4 {
namespace {

template <bool kNv, bool kDown, int kBlocks>
__global__ void __launch_bounds__(kThreads, 1) moe_decode_fp4_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_dyn[];
  Common& c = common_of(smem_dyn);
  prepare(p, c);
  if (kDown) launch_dependents();
  grid_dependency_wait();
  if (!kDown) launch_dependents();
  layer<kNv ? W4_FMT_NVFP4 : W4_FMT_MXFP4, kDown, kBlocks, false>(p, c);
}

template <bool kNv, bool kDown>
cudaError_t run_fitting(const MoeDecodeArgs& a, cudaStream_t s) {
  constexpr int kFmt = kNv ? W4_FMT_NVFP4 : W4_FMT_MXFP4;
  if (a.route.T > 8) return run<moe_decode_fp4_kernel<kNv, kDown, kDown ? 4 : 2>, kFmt, kDown>(a, s);
  if (kDown && a.route.T > 4) return run<moe_decode_fp4_kernel<kNv, kDown, kDown ? 2 : 1>, kFmt, kDown>(a, s);
  return run<moe_decode_fp4_kernel<kNv, kDown, 1>, kFmt, kDown>(a, s);
}

template <bool kNv>
cudaError_t run_both(const MoeDecodeArgs& a, cudaStream_t s) {
  const cudaError_t e = run_fitting<kNv, false>(a, s);
  return e == cudaSuccess ? run_fitting<kNv, true>(a, s) : e;
}

}  // namespace

cudaError_t launch_moe_decode_fp4(const MoeDecodeArgs& a, cudaStream_t s) {
  return a.format == W4_FMT_NVFP4 ? run_both<true>(a, s) : run_both<false>(a, s);
}

}  // namespace w4
