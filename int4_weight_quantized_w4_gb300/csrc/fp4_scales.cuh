// Block scales on their way from rows in memory to the tensor core: 32 bytes of a row at
// a time into shared memory, then, a stage of 256 columns at a time, into atoms of 128 rows'
// 32-bit words (row r's at 16 (r % 32) + 4 (r / 32)), which tcgen05.cp takes.
#pragma once

#include "common.cuh"
#include "tc.cuh"

namespace w4 {
namespace {

constexpr int kStageK = 256;                  // columns of a stage
constexpr int kStageBytes = kStageK / 2;

// By all lanes: 32 bytes of scales of `rows` rows from byte `at` of the row on, those below
// `valid` and SB; zeros elsewhere.
W4_DEV void copy_scale_words(uint32_t to, const uint8_t* src, int SB, int at, int rows, int valid) {
  for (int i = threadIdx.x & 31; i < rows * 8; i += 32) {
    const int r = i >> 3, b = at + 4 * (i & 7);
    const bool in = r < valid && b < SB;
    tc::copy4_async(to + i * 4, in ? src + static_cast<size_t>(r) * SB + b : src, in);
  }
}

// Lane l's words of a stage: rows l, l + 32, l + 64 and l + 96 (those of the first `blocks`
// blocks of 32) from `f`, this lane's first row.
template <bool kNv>
W4_DEV void load_scale_words(const uint8_t* f, int blocks, uint32_t (&v)[4][kNv ? 4 : 2]) {
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if constexpr (kNv) {
      const uint4 x = b < blocks ? *reinterpret_cast<const uint4*>(f + b * 1024) : make_uint4(0, 0, 0, 0);
      v[b][0] = x.x, v[b][1] = x.y, v[b][2] = x.z, v[b][3] = x.w;
    } else {
      const uint2 x = b < blocks ? *reinterpret_cast<const uint2*>(f + b * 1024) : make_uint2(0, 0);
      v[b][0] = x.x, v[b][1] = x.y;
    }
  }
}
// The atoms of the stage's words, `pitch` bytes apart; `to` is this lane's place in the first.
template <bool kNv>
W4_DEV void store_scale_atoms(uint8_t* to, int pitch, const uint32_t (&v)[4][kNv ? 4 : 2]) {
#pragma unroll
  for (int j = 0; j < (kNv ? 4 : 2); ++j) *reinterpret_cast<uint4*>(to + j * pitch) = make_uint4(v[0][j], v[1][j], v[2][j], v[3][j]);
}

}  // namespace
}  // namespace w4
