// One token's choice of experts by a warp, and its weights: the steps that the routing
// kernels and the few-token expert layer share.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace w4 {
namespace {

constexpr uint32_t kNoKey = 0;          // below every key (the key of -inf is 0x007FFFFF)
constexpr unsigned kFull = 0xFFFFFFFFu;

W4_DEV uint32_t ordered_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
W4_DEV float key_value(uint32_t u) { return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }

constexpr float kMaxFinite = 3.402823466e38f;
W4_DEV float sigmoid_f32(float v) { return __frcp_rn(1.f + expf(-v)); }   // 1 / x, correctly rounded

// This lane's logits of token t; lanes and slots past E hold -inf. NaN counts as
// -inf, +inf as the largest finite number.
template <int kEPL>
W4_DEV void load_logits(const MoeRouteArgs& a, int64_t t, float (&v)[kEPL]) {
  const int lane = threadIdx.x & 31;
  bool odd = false;
  if (a.bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(a.logits) + t * a.E + lane;
#pragma unroll
    for (int i = 0; i < kEPL; ++i)
      v[i] = lane + 32 * i < a.E ? __uint_as_float(static_cast<uint32_t>(__ldcg(p + 32 * i)) << 16) : -INFINITY;
  } else {
    const float* p = static_cast<const float*>(a.logits) + t * a.E + lane;
#pragma unroll
    for (int i = 0; i < kEPL; ++i) v[i] = lane + 32 * i < a.E ? __ldcg(p + 32 * i) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < kEPL; ++i) odd |= !(v[i] <= kMaxFinite);
  if (odd) {
#pragma unroll
    for (int i = 0; i < kEPL; ++i) v[i] = isnan(v[i]) ? -INFINITY : fminf(v[i], kMaxFinite);
  }
}

// Chooses for token t with logits v (overwritten). row: kEPL * 33 words of shared
// memory of this warp (expert e at e + e / 32: groups of 32 start in different
// banks). mine: choices lane and lane + 32.
template <int kEPL>
W4_DEV void route_token(const MoeRouteArgs& a, int64_t t, float (&v)[kEPL], uint32_t* row, int (&mine)[2]) {
  const int lane = threadIdx.x & 31;
  const int E = a.E;
  uint32_t key[kEPL];
  float sum = 0.f, mx = -INFINITY;
  if (a.softmax) {
#pragma unroll
    for (int i = 0; i < kEPL; ++i) mx = fmaxf(mx, v[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
  }
  if (a.bias == nullptr) {
#pragma unroll
    for (int i = 0; i < kEPL; ++i) key[i] = lane + 32 * i < E ? ordered_key(v[i]) : kNoKey;
    if (a.softmax) {
#pragma unroll
      for (int i = 0; i < kEPL; ++i) sum += v[i] != -INFINITY ? expf(v[i] - mx) : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    }
  } else {
    if (a.softmax) {
      double d = 0.0;
#pragma unroll
      for (int i = 0; i < kEPL; ++i) {
        v[i] = v[i] != -INFINITY ? expf(v[i] - mx) : 0.f;
        d += static_cast<double>(v[i]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(kFull, d, o);
      sum = static_cast<float>(d);
#pragma unroll
      for (int i = 0; i < kEPL; ++i) v[i] = sum > 0.f ? __fdiv_rn(v[i], sum) : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < kEPL; ++i) v[i] = sigmoid_f32(v[i]);
    }
#pragma unroll
    for (int i = 0; i < kEPL; ++i) {
      const int e = lane + 32 * i;
      key[i] = e < E ? ordered_key(v[i] + a.bias[e]) : kNoKey;
    }
  }

  if (a.topk_group < a.n_group) {
    const int gs = E / a.n_group;
#pragma unroll
    for (int i = 0; i < kEPL; ++i) row[lane + 33 * i] = key[i];
    __syncwarp();
    // L lanes per group (a power of two): lane = group * L + part
    int L = 1;
    while (2 * L * a.n_group <= 32) L *= 2;
    const int g = lane / L;
    uint32_t m1 = kNoKey, m2 = kNoKey;       // the two largest keys of this lane's share
    if (g < a.n_group)
      for (int j = lane & (L - 1); j < gs; j += L) {
        const int e = g * gs + j;
        const uint32_t u = row[e + (e >> 5)];
        m2 = max(m2, min(m1, u));
        m1 = max(m1, u);
      }
    for (int o = 1; o < L; o <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
      m2 = max(max(m2, o2), min(m1, o1));
      m1 = max(m1, o1);
    }
    float gv = key_value(m1);
    if (a.bias != nullptr && gs > 1) gv += key_value(m2);
    const uint32_t gk = ordered_key(isnan(gv) ? -INFINITY : gv);
    int better = 0;
    for (int o = 0; o < a.n_group; ++o) {
      const uint32_t ok = __shfl_sync(kFull, gk, o * L);
      better += ok > gk || (ok == gk && o < g);
    }
    const uint32_t kept = __ballot_sync(kFull, g < a.n_group && better < a.topk_group);   // bit g * L
    const uint32_t magic = ((1u << 20) + gs - 1) / gs;   // e / gs = e * magic >> 20 for e < 1024
#pragma unroll
    for (int i = 0; i < kEPL; ++i) {
      const uint32_t e = lane + 32 * i;
      if (!((kept >> ((e * magic >> 20) * L & 31)) & 1u)) key[i] = kNoKey;
    }
    __syncwarp();
  }
  // the logits, or with a bias the scores, where a choice finds them by expert
#pragma unroll
  for (int i = 0; i < kEPL; ++i) row[lane + 33 * i] = __float_as_uint(v[i]);
  __syncwarp();

  // k rounds of a warp maximum over every lane's best key. b1 and b2 are the
  // lane's two largest, the lower expert first among equals.
  mine[0] = mine[1] = 0;
  uint32_t b1, b2;
  int i1, i2;
  auto scan = [&]() {
    b1 = key[0], i1 = 0, b2 = kNoKey, i2 = 0;
#pragma unroll
    for (int i = 1; i < kEPL; ++i) {
      const bool first = key[i] > b1, second = key[i] > b2;
      b2 = first ? b1 : second ? key[i] : b2;
      i2 = first ? i1 : second ? i : i2;
      b1 = first ? key[i] : b1;
      i1 = first ? i : i1;
    }
  };
  scan();
  uint32_t taken = 0;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t m = __reduce_max_sync(kFull, b1);
    const unsigned e = __reduce_min_sync(kFull, b1 == m ? static_cast<unsigned>(lane + 32 * i1) : 0xFFFFu);
    if (lane == (j & 31)) mine[j >> 5] = static_cast<int>(e);
    if (lane == static_cast<int>(e & 31)) {
      taken |= 1u << i1;
      b1 = b2, i1 = i2, b2 = kNoKey;
      if (kEPL > 1 && b1 == kNoKey) {   // both are taken: look through the rest
#pragma unroll
        for (int i = 0; i < kEPL; ++i)
          if ((taken >> i) & 1u) key[i] = kNoKey;
        scan();
      }
    }
  }
  float w[2], total = 0.f;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    w[s] = 0.f;
    if (lane + 32 * s < a.k) {
      const float x = __uint_as_float(row[mine[s] + (mine[s] >> 5)]);
      if (a.bias != nullptr)
        w[s] = x;
      else if (!a.softmax)
        w[s] = sigmoid_f32(x);
      else
        w[s] = x != -INFINITY ? __fdiv_rn(expf(x - mx), sum) : 0.f;
    }
    total += w[s];
  }
  if (a.renorm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
#pragma unroll
    for (int s = 0; s < 2; ++s) w[s] = total > 0.f ? __fdiv_rn(w[s], total) : 0.f;
  }
#pragma unroll
  for (int s = 0; s < 2; ++s)
    if (lane + 32 * s < a.k) {
      a.ids[t * a.k + lane + 32 * s] = mine[s];
      a.wts[t * a.k + lane + 32 * s] = w[s] * a.factor;
    }
  __syncwarp();   // row is free
}

}  // namespace
}  // namespace w4
