// Grouped routing: sigmoid or softmax scores, a balance bias, expert groups,
// and the expert-sorted row order of the chosen (token, expert) pairs.
//
// The choice goes by a key per expert: the logit, or with a bias fl(score +
// bias). Group values (the largest key, or with a bias the sum of the two
// largest) pick the topk_group best of n_group groups of equal size; the top_k
// largest keys of those are chosen, equal keys and groups in ascending order.
// Weights are the scores, divided by their sum over the chosen when
// renormalizing (0 where that sum is 0), times `factor`.
//
// The steps that decide a choice are fixed to the bit: sigmoid = fl(1 / fl(1 +
// expf(-l))); softmax p = fl(expf(l - max) / S), with S summed in fp64 and
// rounded once when keys depend on it, so that the order of the sum cannot move
// a near-tie.
//
// A warp takes a token: lane l holds experts l, l + 32, ... as integer keys in
// the order of their values (sign folded, -0 taken as +0), so that a warp
// maximum is one redux. A lane keeps its two largest keys at hand and looks
// through the others only when both are taken, which about one of eight choices
// asks for. A CTA takes a tile of tokens and counts its rows per expert; the place
// kernel, a CTA per tile, turns the counts of all tiles into the tile's first row
// in every expert (column sums, then a block scan over the experts) and ranks the
// tile's rows by token with bit masks. At most kMaxTiles tiles, one per SM: the
// count table that every place CTA reads stays small. A call of up to a token per
// warp of one CTA is one launch. Bound by instruction issue for many tokens (1270
// warp instructions a token of 256 experts; 16384 of them 33 us, a quarter of it the
// place kernel), by latency for few (one token 3.9 us, 333 of 96 experts 8). Times are
// GPU times in a CUDA graph of calls.
#include "common.cuh"
#include "launch.h"

namespace w4 {
namespace {

constexpr int kMaxTiles = 152;
constexpr int kChunk = 128;             // tokens ranked at a time
constexpr int kChunkWarps = kChunk / 32;
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
      v[i] = lane + 32 * i < a.E ? __uint_as_float(static_cast<uint32_t>(p[32 * i]) << 16) : -INFINITY;
  } else {
    const float* p = static_cast<const float*>(a.logits) + t * a.E + lane;
#pragma unroll
    for (int i = 0; i < kEPL; ++i) v[i] = lane + 32 * i < a.E ? p[32 * i] : -INFINITY;
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

// Rows of tokens [t0, t1) in order: base[e] is expert e's next row, moved on
// past them. bits, first: [kChunkWarps][E]. All threads of the block take part; a
// thread keeps the experts of its pairs (at most kPairs of a chunk's), `ids` being
// those of the first chunk.
constexpr int kPairs = 8;
struct PairIds {
  int e[kPairs];
};
W4_DEV PairIds load_ids(const MoeRouteArgs& a, int64_t c0, int64_t t1) {
  const int n = static_cast<int>(t1 - c0 < kChunk ? t1 - c0 : kChunk) * a.k;   // pairs of the chunk
  PairIds p;
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    p.e[j] = i < n ? __ldcg(a.ids + c0 * a.k + i) : -1;
  }
  return p;
}
W4_DEV void place_tokens(const MoeRouteArgs& a, int64_t t0, int64_t t1, PairIds ids, uint32_t* bits, int32_t* first,
                         int32_t* base) {
  const int E = a.E, k = a.k;
  for (int64_t c0 = t0; c0 < t1; c0 += kChunk) {
    for (int i = threadIdx.x; i < kChunkWarps * E; i += blockDim.x) bits[i] = 0;
    __syncthreads();
    int tok[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      if (ids.e[j] >= 0) {
        tok[j] = static_cast<int>((threadIdx.x + j * blockDim.x) / static_cast<unsigned>(k));
        ids.e[j] += (tok[j] >> 5) * E;
        atomicOr(&bits[ids.e[j]], 1u << (tok[j] & 31));
      }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      int run = base[e];
      for (int w = 0; w < kChunkWarps; ++w) {
        first[w * E + e] = run;
        run += __popc(bits[w * E + e]);
      }
      base[e] = run;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      if (ids.e[j] >= 0) {
        const int r = first[ids.e[j]] + __popc(bits[ids.e[j]] & ((1u << (tok[j] & 31)) - 1u));
        a.row_token[r] = static_cast<int32_t>(c0 + tok[j]);
        a.row_of[c0 * k + threadIdx.x + j * blockDim.x] = r;
      }
    if (c0 + kChunk < t1) ids = load_ids(a, c0 + kChunk, t1);
    __syncthreads();
  }
}

// base[e] (a count per expert) becomes base[e] + the totals of the experts
// before e; total[e] the expert's rows. Writes offsets when `write`.
W4_DEV void add_expert_starts(const MoeRouteArgs& a, const int32_t* total, int32_t* base, int32_t* part, bool write) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int carry = 0;
  for (int e0 = 0; e0 < a.E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    const int n = e < a.E ? total[e] : 0;
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < nw; ++w) {
      const int v = part[w];
      if (w < warp) before += v;
      carry += v;
    }
    if (e < a.E) {
      base[e] += before + inc - n;
      if (write) a.offsets[e] = before + inc - n;
    }
    __syncthreads();
  }
  if (write && threadIdx.x == 0) a.offsets[a.E] = carry;
}

// Most warps per CTA: the rows of all warps take 34 KB at most.
template <int kEPL>
constexpr int kRouteWarps = kEPL <= 8 ? 32 : 256 / kEPL;
constexpr int kPlaceWords = (2 * kChunkWarps + 2) * 1024;   // bits, first, base, total for 1024 experts

// Tokens [tile * per, ...) of this CTA: choices and weights, then the tile's
// rows per expert into counts[tile][E], or (kWhole: the call is one tile) the
// whole row order.
template <int kEPL, bool kWhole>
__global__ void __launch_bounds__(32 * kRouteWarps<kEPL>) route_tile_kernel(const MoeRouteArgs a, int per,
                                                                           int32_t* __restrict__ counts) {
  constexpr int kKeyWords = kRouteWarps<kEPL> * kEPL * 33;
  __shared__ uint32_t buf[kWhole && kPlaceWords > kKeyWords ? kPlaceWords : kKeyWords];
  __shared__ int32_t cnt[32 * kEPL];
  __shared__ int32_t part[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int e = threadIdx.x; e < 32 * kEPL; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the kernel before writes the logits
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * per, t1 = t0 + per < a.T ? t0 + per : a.T;
  float v[kEPL], next[kEPL];
  if (t0 + warp < t1) load_logits<kEPL>(a, t0 + warp, v);
  for (int64_t t = t0 + warp; t < t1; t += warps) {
    if (!kWhole && t + warps < t1) load_logits<kEPL>(a, t + warps, next);
    int mine[2];
    route_token<kEPL>(a, t, v, buf + warp * kEPL * 33, mine);
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (lane + 32 * s < a.k) atomicAdd(&cnt[mine[s]], 1);
    if (!kWhole) {
#pragma unroll
      for (int i = 0; i < kEPL; ++i) v[i] = next[i];
    }
  }
  __syncthreads();
  if (!kWhole) {
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) counts[static_cast<int64_t>(blockIdx.x) * a.E + e] = cnt[e];
    return;
  }
  int32_t* base = reinterpret_cast<int32_t*>(buf) + 2 * kChunkWarps * a.E;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) base[e] = 0;
  __syncthreads();
  add_expert_starts(a, cnt, base, part, true);
  place_tokens(a, t0, t1, load_ids(a, t0, t1), buf, reinterpret_cast<int32_t*>(buf) + kChunkWarps * a.E, base);
}

// Threads of a place CTA: 1024 for tiles of 64 tokens and more, 512 below (333
// tokens of 96 experts: 7.3 us against 10.5; 16384 of 256: 37 us against 32).
constexpr int kPlaceThreads = 1024;
static_assert(kChunk * 64 <= kPairs * kPlaceThreads && 64 * 64 <= kPairs * 512, "a chunk's pairs at the largest top_k");
__global__ void __launch_bounds__(kPlaceThreads) place_kernel(const MoeRouteArgs a, int per,
                                                              const int32_t* counts, int ntiles) {
  extern __shared__ uint32_t sm[];
  __shared__ int32_t part[kPlaceThreads / 32];
  uint32_t* bits = sm;
  int32_t* first = reinterpret_cast<int32_t*>(sm) + kChunkWarps * a.E;
  int32_t* base = first + kChunkWarps * a.E;
  int32_t* total = base + a.E;
  const int tile = blockIdx.x;
  for (int e = threadIdx.x; e < 2 * a.E; e += blockDim.x) base[e] = 0;   // and total
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t t0 = static_cast<int64_t>(tile) * per, t1 = t0 + per < a.T ? t0 + per : a.T;
  const PairIds ids = load_ids(a, t0, t1);   // on their way during the sums
  // column sums: as many threads per expert as there are, each over a share of the tiles
  const int threads = blockDim.x;
  const int segs = a.E < threads ? threads / a.E : 1;
  const int seg = a.E < threads ? threadIdx.x / a.E : 0;
  if (seg < segs)
    for (int e = threadIdx.x - seg * a.E; e < a.E; e += threads) {
      const int i0 = ntiles * seg / segs, i1 = ntiles * (seg + 1) / segs;
      int before = 0, all = 0;
#pragma unroll 16
      for (int i = i0; i < i1; ++i) {
        const int c = __ldcg(counts + static_cast<int64_t>(i) * a.E + e);
        all += c;
        before += i < tile ? c : 0;
      }
      atomicAdd(&base[e], before);
      atomicAdd(&total[e], all);
    }
  __syncthreads();
  add_expert_starts(a, total, base, part, tile == 0);
  place_tokens(a, t0, t1, ids, bits, first, base);
}

int route_warps(int E) { return E <= 256 ? 32 : E <= 512 ? 16 : 8; }
// One CTA does the whole call up to a token per warp.
bool one_tile(int64_t T, int E) { return T <= route_warps(E); }
// Tokens per tile, at least 4 (a CTA of 4 warps).
int64_t tile_tokens(int64_t T) {
  const int64_t per = (T + kMaxTiles - 1) / kMaxTiles;
  return per < 4 ? 4 : per;
}

template <int kEPL>
cudaError_t launch_k(const MoeRouteArgs& a, cudaStream_t s) {
  if (one_tile(a.T, a.E)) {
    const int warps = a.T < 8 ? 8 : static_cast<int>(a.T);   // ranking and scanning take the whole CTA
    PdlLaunch pl(1, 32 * warps, 0, s);
    return cudaLaunchKernelEx(&pl.cfg, route_tile_kernel<kEPL, true>, a, static_cast<int>(a.T),
                              static_cast<int32_t*>(nullptr));
  }
  const int64_t per = tile_tokens(a.T);
  const int ntiles = static_cast<int>((a.T + per - 1) / per);
  const int warps = static_cast<int>(per < kRouteWarps<kEPL> ? per : kRouteWarps<kEPL>);
  int32_t* counts = static_cast<int32_t*>(a.workspace);
  PdlLaunch rl(ntiles, 32 * warps, 0, s);
  cudaError_t e = cudaLaunchKernelEx(&rl.cfg, route_tile_kernel<kEPL, false>, a, static_cast<int>(per), counts);
  if (e != cudaSuccess) return e;
  PdlLaunch pl(ntiles, per >= 64 ? kPlaceThreads : 512, static_cast<size_t>(2 * kChunkWarps + 2) * a.E * 4, s);   // at most 40 KB
  return cudaLaunchKernelEx(&pl.cfg, place_kernel, a, static_cast<int>(per), static_cast<const int32_t*>(counts), ntiles);
}

}  // namespace

size_t moe_route_grouped_workspace_bytes(int64_t T, int32_t E) {
  if (one_tile(T, E)) return 0;
  const int64_t per = tile_tokens(T);
  return static_cast<size_t>((T + per - 1) / per) * static_cast<size_t>(E) * sizeof(int32_t);
}

cudaError_t launch_moe_route_grouped(const MoeRouteArgs& a, cudaStream_t s) {
  if (a.E <= 32) return launch_k<1>(a, s);
  if (a.E <= 64) return launch_k<2>(a, s);
  if (a.E <= 128) return launch_k<4>(a, s);
  if (a.E <= 256) return launch_k<8>(a, s);
  if (a.E <= 512) return launch_k<16>(a, s);
  return launch_k<32>(a, s);
}

}  // namespace w4
