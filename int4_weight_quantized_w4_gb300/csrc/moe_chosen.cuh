// The chosen experts of a few tokens, in a CTA's shared memory: what the kernels of the
// few-token expert layer share.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "route.cuh"

namespace w4 {
namespace {

constexpr int kMaxT = kMoeDecodeTokens, kMaxE = kMoeDecodeExperts, kMaxK = kMoeDecodeTopK, kMaxPairs = kMaxT * kMaxK;

// What routing leaves: rows of the activations are the chosen pairs by expert, then token.
struct alignas(16) Choice {
  float weight[kMaxPairs];     // of a row
  float x_scale[kMaxT];        // what undoes the factor that brought x_t into range
  int16_t expert[kMaxE];       // the chosen experts in ascending order
  int16_t first[kMaxE + 8];    // their first rows, and behind the last one's
  uint8_t token[kMaxPairs];    // of a row
  int n;                       // how many experts
  int pad[11];
};
static_assert(sizeof(Choice) == kMoeChoiceBytes, "a workspace begins with one");

// In shared memory, the same in every CTA.
struct Routed : Choice {
  uint32_t mask[kMaxE];        // tokens of an expert
  int32_t ids[kMaxPairs];
  float wts[kMaxPairs];
};

// The choice from one kernel to the next, in global memory. All threads.
template <int kThreads>
W4_DEV void keep_choice(const Routed& s, uint4* to) {
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(Choice) / 16); i += kThreads)
    to[i] = reinterpret_cast<const uint4*>(static_cast<const Choice*>(&s))[i];
}
template <int kThreads>
W4_DEV void take_choice(Routed& s, const uint4* from) {
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(Choice) / 16); i += kThreads)
    reinterpret_cast<uint4*>(static_cast<Choice*>(&s))[i] = ld_cg_v4(from + i);
  __syncthreads();
}

template <int kEPL>
W4_DEV void choose(const MoeRouteArgs& a, int t, Routed& s, uint32_t* scratch) {
  int mine[2];
  float v[kEPL];
  load_logits<kEPL>(a, t, v);
  route_token<kEPL>(a, t, v, scratch, mine);
  if (static_cast<int>(threadIdx.x & 31) < a.k) atomicOr(&s.mask[mine[0]], 1u << t);
}

// Before route_all, and before what it reads is there.
template <int kThreads>
W4_DEV void route_prepare(Routed& s) {
  for (int e = threadIdx.x; e < kMaxE; e += kThreads) s.mask[e] = 0;
  __syncthreads();
}

// All kThreads threads. scratch: 8 x 33 words of shared memory a warp. Warps call also(warp) on
// the way. Each CTA does this once, with its instructions not in the cache yet, so that loops
// off the choice itself stay loops.
template <int kThreads, class Also>
W4_DEV void route_all(const MoeRouteArgs& route, Routed& s, uint32_t* scratch, Also also) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = static_cast<int>(route.T), E = route.E, k = route.k;
  for (int t = warp; t < T; t += kThreads / 32) {
    MoeRouteArgs a = route;
    a.ids = s.ids;
    a.wts = s.wts;
    if (E <= 64)
      choose<2>(a, t, s, scratch + warp * 8 * 33);
    else if (E <= 128)
      choose<4>(a, t, s, scratch + warp * 8 * 33);
    else
      choose<8>(a, t, s, scratch + warp * 8 * 33);
  }
  also(warp);
  __syncthreads();
  // the chosen experts and their first rows, 32 experts at a time
  if (warp == 0) {
    int n = 0, rows = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < E; e0 += 32) {
      const uint32_t m = s.mask[e0 + lane];
      const uint32_t some = __ballot_sync(kFull, m != 0);
      int inc = __popc(m);
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += u;
      }
      const int first = rows + inc - __popc(m);
      if (m != 0) {
        const int i = n + __popc(some & ((1u << lane) - 1u));
        s.expert[i] = static_cast<int16_t>(e0 + lane);
        s.first[i] = static_cast<int16_t>(first);
        s.mask[e0 + lane] = m | static_cast<uint32_t>(first) << 16;   // for the rows below
      }
      n += __popc(some);
      rows += __shfl_sync(kFull, inc, 31);
    }
    if (lane == 0) {
      s.n = n;
      s.first[n] = static_cast<int16_t>(rows);
    }
  }
  __syncthreads();
#pragma unroll 1
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
