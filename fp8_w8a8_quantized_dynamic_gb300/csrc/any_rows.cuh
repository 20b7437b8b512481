// Rows of 16-bit values that start and end anywhere, eight values at a time in whole 16-byte pieces.
#pragma once

#include "device_common.cuh"

namespace fp8k {

// (not through the read-only path: rows may be written over)
__device__ __forceinline__ uint4 load_piece(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Sixteen values a (low), b: the eight from the at-th on, at < 8.
__device__ __forceinline__ uint4 eight_from(uint4 a, uint4 b, int at) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = at & 4 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = at & 2 ? w[i + 1] : w[i];
  const int bits = at & 1 ? 16 : 0;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// The first n values of v, zeros behind them.
__device__ __forceinline__ uint4 first_of(uint4 v, int n) {
  auto keep = [&](uint32_t w, int i) { return i + 1 < n ? w : i < n ? w & 0xFFFFu : 0u; };
  return make_uint4(keep(v.x, 0), keep(v.y, 2), keep(v.z, 4), keep(v.w, 6));
}

// Values c .. c + 7 of a row, c < cols, zeros from cols on: from the one or two whole pieces that hold them. Each of those
// holds one of the row's values, so that all of it may be read.
__device__ __forceinline__ uint4 load8_any(const uint16_t* row, int64_t c, int64_t cols) {
  const uint16_t* first = row + c;
  const int at = int(reinterpret_cast<uintptr_t>(first) >> 1) & 7;
  const uint4* piece = reinterpret_cast<const uint4*>(first - at);
  const int n = int(cols - c < 8 ? cols - c : 8);
  const uint4 a = load_piece(piece);
  if (at == 0) return n < 8 ? first_of(a, n) : a;
  const uint4 b = at + n > 8 ? load_piece(piece + 1) : make_uint4(0, 0, 0, 0);
  const uint4 v = eight_from(a, b, at);
  return n < 8 ? first_of(v, n) : v;
}

// load8_any in two halves, for loads that run ahead of their use: the pieces, and the values in them. `at` = off_piece(row + c).
struct Raw8 {
  uint4 a, b;
};
__device__ __forceinline__ int off_piece(const uint16_t* p) { return int(reinterpret_cast<uintptr_t>(p) >> 1) & 7; }
__device__ __forceinline__ Raw8 load8_raw(const uint16_t* row, int at, int c, int cols) {
  Raw8 v;
  v.a = v.b = make_uint4(0, 0, 0, 0);
  const uint4* piece = reinterpret_cast<const uint4*>(row + c - at);
  if (c < cols) v.a = load_piece(piece);
  if (at != 0 && c - at + 8 < cols) v.b = load_piece(piece + 1);
  return v;
}
__device__ __forceinline__ uint4 values8(const Raw8& v, int at, int c, int cols) {
  uint4 e = v.a;
  if (at != 0) e = eight_from(v.a, v.b, at);
  // (c + 8 passes 31 bits in rows of almost 2^31 columns; c itself may behind a row, where v is zeros)
  if (c > cols - 8) e = first_of(e, cols > c ? cols - c : 0);
  return e;
}

// Values [from, to) of eight to their places in a piece. Those of a piece's end or start take three stores of 8, 4 and 2 bytes
// at most: by values, the two ends of a warp's run take as long as all else of it (the gradient of 16384 x 4095, one row a token:
// 161 us, 127 so).
__device__ __forceinline__ void store_some(uint16_t* piece, uint4 v, int from, int to) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  auto word = [&](int i) { return i & 2 ? (i & 1 ? v.w : v.z) : (i & 1 ? v.y : v.x); };
  if (from == 0) {
    if (to & 8) *reinterpret_cast<uint4*>(piece) = v;
    if (to & 4) *reinterpret_cast<uint2*>(piece) = make_uint2(v.x, v.y);
    if (to & 2) *reinterpret_cast<uint32_t*>(piece + (to & 4)) = word((to & 4) >> 1);
    if (to & 1) piece[to - 1] = uint16_t(word(to >> 1));
  } else if (to == 8) {
    if (from & 1) piece[from] = uint16_t(word(from >> 1) >> 16);
    if ((8 - from) & 2) *reinterpret_cast<uint32_t*>(piece + (from < 4 ? 2 : 6)) = from < 4 ? v.y : v.w;
    if (from <= 4) *reinterpret_cast<uint2*>(piece + 4) = make_uint2(v.z, v.w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= from && i < to) piece[i] = uint16_t(w[i >> 1] >> (16 * (i & 1)));
  }
}
// The last values of eight, from the from-th on, to the start of a piece: n of them at most.
__device__ __forceinline__ void store_rest(uint16_t* piece, uint4 v, int from, int n) {
  if (n > 0) store_some(piece, eight_from(v, make_uint4(0, 0, 0, 0), from), 0, n);
}

// Stores values c .. c + 7 of a row (those before cols): all lanes of the warp come here, `live` ones have some. Where a lane is
// joined, the lane before it has the eight before its own; where it hands on, the lane after it is joined. A lane stores the
// whole piece that ends with its own values, with what it takes from the lane before; the ends of a run of lanes are stored in
// parts.
__device__ __forceinline__ void store8_run(uint16_t* row, int64_t c, int64_t cols, uint4 v, bool live, bool joined,
                                           bool handed_on) {
  uint4 before;
  before.x = __shfl_up_sync(0xffffffffu, v.x, 1);
  before.y = __shfl_up_sync(0xffffffffu, v.y, 1);
  before.z = __shfl_up_sync(0xffffffffu, v.z, 1);
  before.w = __shfl_up_sync(0xffffffffu, v.w, 1);
  if (!live) return;
  uint16_t* first = row + c;
  const int at = off_piece(first);  // values of the piece that lie before c
  const int n = int(cols - c < 8 ? cols - c : 8);
  if (at == 0) {
    if (n == 8)
      *reinterpret_cast<uint4*>(first) = v;
    else
      store_some(first, v, 0, n);
    return;
  }
  const uint4 piece = eight_from(before, v, 8 - at);
  if (joined && at + n >= 8)
    *reinterpret_cast<uint4*>(first - at) = piece;
  else
    store_some(first - at, piece, joined ? 0 : at, at + n < 8 ? at + n : 8);
  if (!handed_on) store_rest(first - at + 8, v, 8 - at, at + n - 8);
}
// The same for sixteen values a lane, lo and hi.
__device__ __forceinline__ void store16_run(uint16_t* row, int64_t c, int64_t cols, uint4 lo, uint4 hi, bool live, bool joined,
                                            bool handed_on) {
  uint4 before;
  before.x = __shfl_up_sync(0xffffffffu, hi.x, 1);
  before.y = __shfl_up_sync(0xffffffffu, hi.y, 1);
  before.z = __shfl_up_sync(0xffffffffu, hi.z, 1);
  before.w = __shfl_up_sync(0xffffffffu, hi.w, 1);
  if (!live) return;
  uint16_t* first = row + c;
  const int at = off_piece(first);
  const int n = int(cols - c < 16 ? cols - c : 16);
  if (at != 0) {
    const uint4 piece = eight_from(before, lo, 8 - at);
    if (joined && at + n >= 8)
      *reinterpret_cast<uint4*>(first - at) = piece;
    else
      store_some(first - at, piece, joined ? 0 : at, at + n < 8 ? at + n : 8);
    lo = eight_from(lo, hi, 8 - at);
    first += 8 - at;
  }
  // now lo holds the values from `first` on; the last `at` of hi go to the next lane
  const int left = n - (at != 0 ? 8 - at : 0);
  if (left >= 8)
    *reinterpret_cast<uint4*>(first) = lo;
  else
    store_some(first, lo, 0, left > 0 ? left : 0);
  if (at == 0) {
    if (n == 16)
      *reinterpret_cast<uint4*>(first + 8) = hi;
    else
      store_some(first + 8, hi, 0, n > 8 ? n - 8 : 0);
  } else if (!handed_on) {
    store_rest(row + c - at + 16, hi, 8 - at, at + n - 16);
  }
}

// Lanes with consecutive eights of rows, one row after the other.
__device__ __forceinline__ void store8_any(uint16_t* row, int64_t c, int64_t cols, uint4 v, bool live) {
  const int lane = threadIdx.x & 31;
  store8_run(row, c, cols, v, live, lane > 0 && c > 0, lane < 31 && c + 8 < cols);
}

}  // namespace fp8k
