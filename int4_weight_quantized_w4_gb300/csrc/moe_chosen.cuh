// The chosen experts of a few tokens, in a CTA's shared memory: what the kernels of the
// few-token expert layer share.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "route.cuh"

namespace w4 {
namespace {

constexpr int kMaxT = kMoeDecodeTokens, kMaxE = kMoeDecodeExperts, kMaxK = kMoeDecodeTopK, kMaxPairs = kMaxT * kMaxK;

// What routing leaves in shared memory, the same in every CTA. Rows of the activations
// are the chosen pairs by expert, then token.
struct Routed {
  uint32_t mask[kMaxE];        // tokens of an expert
  int32_t ids[kMaxPairs];
  float wts[kMaxPairs];
  float weight[kMaxPairs];     // of a row
  uint8_t token[kMaxPairs];    // of a row
  int16_t expert[kMaxE];       // the chosen experts in ascending order
  int16_t first[kMaxE + 1];    // their first rows
  int32_t part[8];
  int n;                       // how many
  int x_exp[kMaxT];            // exponent taken out of x_t
};

// All kThreads (at least 256) threads. scratch: 8 x 33 words of shared memory a warp. Warps
// call also(warp) on the way.
template <int kThreads, class Also>
W4_DEV void route_all(const MoeRouteArgs& route, Routed& s, uint32_t* scratch, Also also) {
  static_assert(kThreads >= 256, "a thread to an expert");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = static_cast<int>(route.T), E = route.E, k = route.k;
  for (int e = threadIdx.x; e < kMaxE; e += kThreads) s.mask[e] = 0;
  __syncthreads();
  for (int t = warp; t < T; t += kThreads / 32) {
    MoeRouteArgs a = route;
    a.ids = s.ids;
    a.wts = s.wts;
    int mine[2];
    if (E <= 64) {
      float v[2];
      load_logits<2>(a, t, v);
      route_token<2>(a, t, v, scratch + warp * 8 * 33, mine);
    } else {
      float v[8];
      load_logits<8>(a, t, v);
      route_token<8>(a, t, v, scratch + warp * 8 * 33, mine);
    }
    if (lane < k) atomicOr(&s.mask[mine[0]], 1u << t);
  }
  also(warp);
  __syncthreads();
  // the chosen experts and their first rows: a scan of (rows, experts) over 256 threads
  int v = 0, inc = 0;
  if (warp < 8) {
    const uint32_t m = s.mask[threadIdx.x];
    v = inc = m != 0 ? (__popc(m) << 16) | 1 : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) s.part[warp] = inc;
  }
  __syncthreads();
  if (warp < 8) {
    int before = inc - v;
    for (int w = 0; w < warp; ++w) before += s.part[w];
    if (v != 0) {
      s.expert[before & 0xFFFF] = static_cast<int16_t>(threadIdx.x);
      s.first[before & 0xFFFF] = static_cast<int16_t>(before >> 16);
      s.mask[threadIdx.x] |= (before >> 16) << 16;   // first row beside the tokens, for the rows below
    }
    if (threadIdx.x == 255) {
      s.n = (before + v) & 0xFFFF;
      s.first[s.n] = static_cast<int16_t>((before + v) >> 16);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < T * k; i += kThreads) {
    const uint32_t m = s.mask[s.ids[i]];
    const int t = i / k, r = static_cast<int>(m >> 16) + __popc(m & 0xFFFFu & ((1u << t) - 1u));
    s.token[r] = static_cast<uint8_t>(t);
    s.weight[r] = s.wts[i];
  }
  __syncthreads();
}

}  // namespace
}  // namespace w4
