// parts.h -- into how many parts the products of the checkpointed expert backward
// are cut where their tiles are too few for the GPU, and the room that their
// FP32 outputs take.  Host arithmetic; sms is the device's number of SMs.
#pragma once

#include <algorithm>
#include <cstdint>

namespace moe {
namespace parts {

// Tiles are 128 rows, or 256 on CTA pairs, by 256 columns; a k-block is 64 deep.
constexpr int64_t kRows = 128, kCols = 256, kDepth = 64;

inline int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

// Parts that each expert's rows are cut into for a weight gradient of m x n:
// one, or as many as fill the CTA pairs where the tiles of all experts are
// fewer, with four k-blocks a part at least on average (below that the parts'
// FP32 outputs cost more than they save).  Two experts of 664 x 112 with 10280
// rows each: 185 us with one part.
inline int weight_gradient(int64_t N, int64_t E, int64_t m, int64_t n, int64_t sms) {
  const int64_t tiles = E * tiles_of(m, 2 * kRows) * tiles_of(n, kCols);
  return (int)std::max<int64_t>(1, std::min(sms / 2 / tiles, N / (E * 4 * kDepth)));
}

// Parts that dinput's K = 2 I is cut into where its tiles are fewer than the SMs
// (few rows, H short): as many as fill them, of eight k-blocks at least.  A
// captured backward of 30 rows over five experts of 696 x 3688 takes 86 us,
// 135 with one part; of 1 row of 64 x 512, the smallest that is cut, 41 and 46.
inline int64_t most_of_depth(int64_t I) { return 2 * tiles_of(I, kDepth) / 8; }
inline int dinput(int64_t N, int64_t E, int64_t H, int64_t I, int64_t sms) {
  const bool pair = N >= kRows * E;
  const int64_t mt = N / (pair ? 2 * kRows : kRows) + std::min(E, N);
  const int64_t tiles = std::max<int64_t>(1, mt * tiles_of(H, kCols));
  return (int)std::max<int64_t>(1, std::min((pair ? sms / 2 : sms) / tiles, most_of_depth(I)));
}

// FP32 values that the parts of a batch of up to N rows take: this does not fall
// as N grows, though the parts of dinput do, so that a workspace made for N rows
// serves fewer.  Parts and tiles of dinput together fill the SMs at most, so
// its outputs are no more than so many tiles (N < 128 mt, or 256 mt on half as
// many pairs); nor more than the parts that its depth allows.
inline int64_t room(int64_t N, int64_t E, int64_t H, int64_t I, int64_t sms) {
  const int64_t gate_up = weight_gradient(N, E, 2 * I, H, sms), down = weight_gradient(N, E, H, I, sms);
  const int64_t weights = std::max(gate_up > 1 ? 2 * gate_up : 0, down > 1 ? down : 0) * E * I * H;
  const int64_t most = std::min(sms / tiles_of(H, kCols), most_of_depth(I));
  return std::max(weights, most > 1 ? std::min(most * N * H, sms * kRows * kCols) : 0);
}

}  // namespace parts
}  // namespace moe
