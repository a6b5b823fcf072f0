// Which rows a block of the linear-attention kernels walks: whole grids, or
// the segments of a call that splits its grids along the rows.
#pragma once

#include "tb_seq.h"

namespace tb {

struct LinSegment {
  int grid;          // -1: the slot holds no segment
  int slot;
  int index, count;  // of the grid's segments
  int64_t begin, end;  // the grid's rows
  int64_t first;     // the segment's places in the order of the walk: [first, first + len)
  int len;
};

__device__ __forceinline__ void lin_grid_rows(const LinLaunch& l, int b, int64_t& begin, int64_t& end) {
  if (!l.offsets) {
    begin = 0;
    end = l.tokens;
    return;
  }
  begin = min(max(l.offsets[b], (int64_t)0), l.tokens);
  end = min(max(l.offsets[b + 1], begin), l.tokens);
}

// The rows that grids have are [begin, end): those before the first offset and
// past the last one belong to none.
struct LinCover {
  int64_t begin, end;
};
__device__ __forceinline__ LinCover lin_cover(const LinLaunch& l) {
  if (!l.offsets) return {0, l.tokens};
  const int64_t begin = min(max(l.offsets[0], (int64_t)0), l.tokens);
  return {begin, min(max(l.offsets[l.grids], begin), l.tokens)};
}

// Zeros for the output rows [r0, r1) of `heads` heads from h on, by `threads`
// threads of which this is number `rank`, counting the rows that no grid has:
// row r is row r of the call, past the cover's begin row r - begin + end.
// E: any type of the outputs' size.
template <class E>
__device__ __noinline__ void lin_zero_rows(const LinProblem& p, LinCover c, int64_t r0, int64_t r1, int h, int heads,
                                           int rank, int threads) {
  constexpr int kVec = 16 / (int)sizeof(E);
  const bool vec = ((uintptr_t)p.out & 15) == 0 && p.o_row % kVec == 0 && p.o_head % kVec == 0 && p.V % kVec == 0;
  const int units = vec ? p.V / kVec : p.V;  // of a row's head; as many rows at a time as the threads take
  const int many = threads / units, step = many ? units : threads;
  if (many && rank >= many * units) return;
  for (int64_t r = r0 + (many ? rank / units : 0); r < r1; r += many ? many : 1) {
    E* to = (E*)p.out + (r < c.begin ? r : r - c.begin + c.end) * p.o_row + h * p.o_head;
    for (int i = 0; i < heads; ++i, to += p.o_head)
      for (int at = rank % step; at < units; at += step) {
        if (vec) *reinterpret_cast<uint4*>(to + at * kVec) = make_uint4(0u, 0u, 0u, 0u);
        else to[at] = E(0);
      }
  }
}
// A slot's share of all of them, in the kernel's prologue by warps that have no
// part in it: calls whose offsets cover the rows take as long as before (32
// grids of 2048 rows, 16 heads of 64 in bf16: 105 us), a buffer of 131072 rows
// of 16 heads of 128 that holds one grid of 65536 358 us, 270 with its 268 MB of
// other rows left alone.
template <class E>
__device__ __forceinline__ void lin_zero_share(const LinLaunch& l, const LinProblem& p, int slot, int h, int heads, int rank,
                                               int threads) {
  const LinCover c = lin_cover(l);
  const int64_t rows = c.begin + l.tokens - c.end;
  if (rows == 0) return;
  const int64_t per = (rows + l.segments - 1) / l.segments, r0 = min(slot * per, rows);
  lin_zero_rows<E>(p, c, r0, min(r0 + per, rows), h, heads, rank, threads);
}
template <int size> struct LinBits { typedef uint16_t type; };
template <> struct LinBits<4> { typedef uint32_t type; };

__device__ __forceinline__ int lin_segments_of(const LinLaunch& l, int64_t rows) {
  return rows > 0 ? (int)((rows + l.segment - 1) / l.segment) : 1;
}

// The segment slot of grid b's first segment.  One warp; the same in all lanes.
__device__ __forceinline__ int lin_first_slot(const LinLaunch& l, int b) {
  int sum = 0;
  for (int i = threadIdx.x & 31; i < b; i += 32) {
    int64_t begin, end;
    lin_grid_rows(l, i, begin, end);
    sum += lin_segments_of(l, end - begin);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

// The segment of a slot, found by one warp; the same in all lanes.
__device__ __forceinline__ LinSegment lin_segment(const LinLaunch& l, int slot) {
  LinSegment s;
  s.grid = -1;
  s.slot = slot;
  s.len = 0;
  if (l.segment == 0) {
    s.grid = slot;
    s.index = 0;
    s.count = 1;
    lin_grid_rows(l, slot, s.begin, s.end);
    s.first = 0;
    s.len = (int)(s.end - s.begin);
    return s;
  }
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int base = 0; base < l.grids; base += 32) {
    int64_t begin = 0, end = 0;
    int n = 0;
    if (base + lane < l.grids) {
      lin_grid_rows(l, base + lane, begin, end);
      n = lin_segments_of(l, end - begin);
    }
    int upto = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + upto > slot);
    if (hit) {
      const int src = __ffs(hit) - 1;
      s.grid = base + src;
      s.count = __shfl_sync(0xffffffffu, n, src);
      s.index = slot - before - __shfl_sync(0xffffffffu, upto - n, src);
      s.begin = __shfl_sync(0xffffffffu, begin, src);
      s.end = __shfl_sync(0xffffffffu, end, src);
      s.first = (int64_t)s.index * l.segment;
      s.len = (int)min((int64_t)l.segment, s.end - s.begin - s.first);
      return s;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return s;
}

// The grid that has `rank` longer ones (ties: the lower index first), of at
// most kLinMaxSorted grids.  One warp; the same in all lanes.  Every block
// does it, so it is short: 32 bits, eight shuffles in flight (64
// grids of 32 rows, 8 heads of 128 x 128, 512 blocks: 29 us, 25 unsorted).
__device__ __forceinline__ int lin_grid_of_rank(const LinLaunch& l, int rank) {
  const int lane = threadIdx.x & 31;
  int rows[kLinMaxSorted / 32], ahead[kLinMaxSorted / 32], found = 0;
#pragma unroll
  for (int i = 0; i < kLinMaxSorted / 32; ++i) {
    rows[i] = -1;
    ahead[i] = 0;
    if (32 * i + lane < l.grids) {
      int64_t begin, end;
      lin_grid_rows(l, 32 * i + lane, begin, end);
      rows[i] = (int)(end - begin);
    }
  }
#pragma unroll
  for (int j = 0; j < kLinMaxSorted / 32; ++j)
#pragma unroll 1
    for (int k0 = 0; k0 < 32 && 32 * j + k0 < l.grids; k0 += 8)
#pragma unroll
      for (int k = k0; k < k0 + 8; ++k) {  // of the lanes without a grid, -1 is ahead of none
        const int x = __shfl_sync(0xffffffffu, rows[j], k);
#pragma unroll
        for (int i = 0; i < kLinMaxSorted / 32; ++i) ahead[i] += x + (32 * j + k < 32 * i + lane) > rows[i];
      }
#pragma unroll
  for (int i = 0; i < kLinMaxSorted / 32; ++i) {
    const unsigned hit = __ballot_sync(0xffffffffu, 32 * i + lane < l.grids && ahead[i] == rank);
    if (hit) found = 32 * i + __ffs(hit) - 1;
  }
  return found;
}

// decay^n for n >= 0.  The logarithm's relative error of 2^-24 moves the
// result by n |log2 decay| 2^-24, which is small wherever the power is not.
__device__ __forceinline__ float lin_power(float decay, float n) {
  return n > 0.f ? exp2f(n * log2f(decay)) : 1.f;
}

}  // namespace tb
