// product_lanes.h -- which 16 bytes of a row of K values a lane loads where rows come
// straight to registers (product8_rows_kernel in product.hip).  Plain C++, so that a host
// program can check that every one of them is inside its row.
#pragma once

namespace gdr {

constexpr int kBlock = 128;  // values of a row that share a scale

// Of block b a lane with lane / 16 = q takes 16 values from 128 b + 16 q on (half 0) and 16
// from 128 b + 64 + 16 q on (half 1).
constexpr int lane_start(int b, int q, int half) { return b * kBlock + half * 64 + q * 16; }

// Whether the row has them: K is a multiple of 16, so it has all 16 or none.
constexpr bool lane_has(int K, int b, int q, int half) { return lane_start(b, q, half) < K; }

// Where in its row the lane loads: the row's first 16 where it has no others, which every row
// has (K >= 16); they are taken for zeros when they are used.
constexpr int lane_offset(int K, int b, int q, int half) {
  return lane_has(K, b, q, half) ? lane_start(b, q, half) : 0;
}

}  // namespace gdr
