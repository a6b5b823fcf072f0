// What the kernels of the selective scan share: how a warp's lanes hold a tile
// of channels and states, rows through shared memory, the functions of a step.
//
// A warp takes the rows of a tile of channels and of up to 16 states, a lane 4
// of the channels and NN of the states: a row costs it one 16-byte read each of
// delta and delta x, and NN numbers each of b and c, for 4 NN updates of h.  The
// walks (tb_scan.cu) hold 64 channels, two lanes to a channel's states, the
// gradient (tb_scan_backward.cu), which keeps four rows' states at once, 32
// channels and four lanes.  Sums over states or channels are a lane's own first
// and then go through shared memory: a lane writes its part, and the lane of a
// channel (or state) reads and adds what belongs to it.
//
// Issued instructions, exponentials and multiply-adds are each about half of a
// walk's time, so numbers go in pairs, two to an instruction (fma.rn.f32x2).  What belongs to a row and a channel (steps, gates, outputs)
// is done by pairs of channels as well.
#pragma once

#include "tb_linattn.cuh"
#include "tb_seq.cuh"

#include <cfloat>

namespace tb {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// --------------------------------------------------------- functions of a step

__device__ __forceinline__ float scan_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float scan_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// a log2(e), finite where a is minus infinity (a channel without memory): the
// rows past a segment's end in its last tile take steps of zero, whose decay is 1.
__device__ __forceinline__ float scan_rate(float a) {
  const float a2 = a * kLog2e;
  return a2 < -FLT_MAX ? -FLT_MAX : a2;
}
// exp(delta a) for a2 = scan_rate(a).  The instruction rounds towards zero: over
// [-1, 0] its results are 2e-8 to 5e-8 low on average (measured), which the
// many decays that a slow state goes through would add up.  2^-25 more in the
// exponent takes most of that back, and costs nothing as a sum.
__device__ __forceinline__ float scan_decay(float delta, float a2) { return scan_ex2(fmaf(delta, a2, 0x1p-25f)); }
__device__ __forceinline__ f32x2 scan_decay(f32x2 delta, f32x2 a2) {
  const float2 x = halves(fma2(delta, a2, both(0x1p-25f)));
  return pair(scan_ex2(x.x), scan_ex2(x.y));
}

// exp(delta a) x + own over many rows at once: delta is their sum.  Where a state
// grows, the factor may be beyond 32 bits although the walk row by row is not: x
// is zero, or small.  Past 2^127 x takes the rest of the exponent first, and a
// zero stays one.
constexpr float kMostExponent = 127.f;
__device__ __forceinline__ float scan_exponent(float delta, float a2) { return fmaf(delta, a2, 0x1p-25f); }
__device__ __forceinline__ float scan_exponent(f32x2 delta, f32x2 a2) {  // the larger one
  const float2 e = halves(fma2(delta, a2, both(0x1p-25f)));
  return fmaxf(e.x, e.y);
}
__device__ __forceinline__ float scan_raised(float e, float x) {  // x 2^(e - 127)
  return x == 0.f ? x : x * scan_ex2(e - kMostExponent);
}
__device__ __forceinline__ float scan_carried(float delta, float a2, float x, float own) {
  const float e = scan_exponent(delta, a2);
  if (e > kMostExponent) return fmaf(0x1p127f, scan_raised(e, x), own);
  return fmaf(scan_ex2(e), x, own);
}
__device__ __forceinline__ f32x2 scan_carried(f32x2 delta, f32x2 a2, f32x2 x, f32x2 own) {
  const float2 d = halves(delta), a = halves(a2), f = halves(x), o = halves(own);
  return pair(scan_carried(d.x, a.x, f.x, o.x), scan_carried(d.y, a.y, f.y, o.y));
}

// log(1 + exp(v)) = max(v, 0) + log(1 + u), u = exp(-|v|), and log(1 + u) = 2
// artanh(s), s = u / (2 + u) <= 1/3: small steps keep their relative accuracy.
// artanh(s) = s + s q P(q), q = s^2, with P of degree 3 fitted to its series on
// [0, 1/9]: 6e-9 off at most.
__device__ __forceinline__ f32x2 scan_softplus(f32x2 v) {
  const float2 f = halves(v);
  const f32x2 e = mul2(pair(-fabsf(f.x), -fabsf(f.y)), both(kLog2e));
  const float2 g = halves(e);
  const f32x2 u = pair(scan_ex2(g.x), scan_ex2(g.y));
  const float2 w = halves(add2(u, both(2.f)));
  const f32x2 s = mul2(u, pair(scan_rcp(w.x), scan_rcp(w.y))), q = mul2(s, s);
  f32x2 p = fma2(both(0.14005993f), q, both(0.14000903f));
  p = fma2(p, q, both(0.20010763f));
  p = fma2(p, q, both(0.3333321f));
  const f32x2 l = fma2(mul2(p, q), s, s);
  return fma2(both(2.f), l, pair(fmaxf(f.x, 0.f), fmaxf(f.y, 0.f)));
}
__device__ __forceinline__ float scan_softplus(float v) { return halves(scan_softplus(both(v))).x; }

// At the ends of the range the exponential is 0 or infinite and the quotient 1 or 0.
__device__ __forceinline__ float scan_sigmoid(float v) { return scan_rcp(1.f + scan_ex2(-v * kLog2e)); }
__device__ __forceinline__ f32x2 scan_sigmoid(f32x2 v) {
  const float2 e = halves(mul2(v, both(-kLog2e)));
  const float2 w = halves(add2(pair(scan_ex2(e.x), scan_ex2(e.y)), both(1.f)));
  return pair(scan_rcp(w.x), scan_rcp(w.y));
}

// ------------------------------------------------------------ rows of a tile

__device__ __forceinline__ void copy_row(void* dst, const void* src, int bytes) {  // 16 bytes, zeros past `bytes`
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_on_their_way() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_for_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  __syncwarp();
}

// -------------------------------------------------------- segments of the rows
//
// Grid b's segments have the slots from begin / segment + b on, with begin its
// first row.  They do not meet the next grid's, as ceil(rows / segment) is at
// most the difference of the two quotients and one; and none is past tokens /
// segment + grids - 1, whatever the offsets are.  So a slot's grid is found by
// halving (by 33 parts, a warp's lanes at once), not by adding up the grids
// before it: the gradient of 20000 grids of one row, 1024 channels, took 322 ms
// when every warp did that.
__device__ __forceinline__ int scan_first_slot(const ScanLaunch& l, int b) {
  if (!l.offsets) return 0;
  return (int)((uint32_t)min(max(l.offsets[b], (int64_t)0), l.tokens) / (uint32_t)l.segment) + b;
}
__device__ __forceinline__ int scan_segments_of(const ScanLaunch& l, int64_t rows) {  // a grid without rows has one too
  return rows > 0 ? (int)(((uint32_t)rows - 1) / (uint32_t)l.segment) + 1 : 1;
}
// By one warp, the same in all lanes; whole grids where there are no segments.
__device__ __forceinline__ LinSegment scan_segment_of(const ScanLaunch& l, int slot) {
  LinSegment s;
  s.slot = slot;
  s.grid = -1;
  s.index = 0;
  s.count = 1;
  s.first = 0;
  s.len = 0;
  int lo = slot;
  if (l.segment) {
    int hi = l.grids;  // first slot of lo <= slot < first slot of hi
    lo = -1;
    while (hi - lo > 1) {
      const int64_t step = ((int64_t)hi - lo + 30) / 32, at = lo + ((threadIdx.x & 31) + 1) * step;
      const unsigned past = __ballot_sync(0xffffffffu, at >= hi || scan_first_slot(l, (int)at) > slot);
      const int n = past ? __ffs(past) - 1 : 32;
      hi = (int)min((int64_t)hi, lo + (n + 1) * step);
      lo += (int)(n * step);
    }
    if (lo < 0) return s;
    s.index = slot - scan_first_slot(l, lo);
  }
  lin_grid_rows(l, lo, s.begin, s.end);
  if (l.segment) {
    s.count = scan_segments_of(l, s.end - s.begin);
    if (s.index >= s.count) return s;
    s.first = (int64_t)s.index * l.segment;
  }
  s.grid = lo;
  s.len = (int)(l.segment ? min((int64_t)l.segment, s.end - s.begin - s.first) : s.end - s.begin);
  return s;
}

// The channels of a warp.  The workspace's arrays have group_pad channels for
// each group, its own rounded up to kScanChannels: a tile's place in them is
// whole, and is read and written without a question for its last channels.
struct ScanTile {
  int group, first, count;  // first channel of all; count <= 0: none
  int64_t place;            // first channel in the workspace
};
template <int CH>
__device__ __forceinline__ ScanTile scan_tile(const ScanLaunch& l, int group, int tile) {
  const int per = l.a.channels / l.a.groups;
  return {group, group * per + tile * CH, min(CH, per - tile * CH), (int64_t)group * l.group_pad + tile * CH};
}

// Where the workspace holds the states before tile i >= 1 of the segment that
// starts at row0: as many places as the call has whole tiles, whatever its
// grids.  Segments that follow one another do not meet there: with len rows, the
// last of ceil(len / 8) tiles lies before place (row0 + len) / 8.
__device__ __forceinline__ int64_t scan_tile_place(int64_t row0, int i) { return row0 / kTileRows + i - 1; }

// Rows [row, row + n) of a tile's channels to dst [kTileRows][CH], zeros past
// them; asynchronous where vectors fit.
template <class T, int CH>
__device__ __forceinline__ void scan_fetch(T* dst, const void* src, int64_t stride, int64_t row, int n, const ScanTile& t, bool vec) {
  const int lane = threadIdx.x & 31;
  const T* from = (const T*)src + t.first;
  if (vec && t.count == CH) {
    constexpr int kChunk = 16 / (int)sizeof(T), kPer = CH / kChunk;
#pragma unroll
    for (int k = 0; k < kTileRows * kPer / 32; ++k) {
      const int i = k * 32 + lane, r = i / kPer, c = i % kPer * kChunk;
      copy_row(dst + r * CH + c, from + (row + min(r, max(n - 1, 0))) * stride + c, r < n ? 16 : 0);
    }
  } else {
    for (int r = 0; r < kTileRows; ++r)
#pragma unroll
      for (int c = lane; c < CH; c += 32)
        dst[r * CH + c] = r < n && c < t.count ? from[(row + r) * stride + c] : RowType<T>::from(0.f);
  }
}

// The two channels of a lane in what is done by rows and channels: 2 (lane %
// (CH / 2)), of row lane / (CH / 2) of as many.
template <int CH>
__device__ __forceinline__ int lane_pair() { return (threadIdx.x & 31) % (CH / 2); }
template <int CH>
__device__ __forceinline__ int lane_row() { return (threadIdx.x & 31) / (CH / 2); }
template <class T, int CH>
__device__ __forceinline__ f32x2 row_pair(const T (&row)[CH]) {
  const int p = lane_pair<CH>();
  if constexpr (sizeof(T) == 4) {
    return reinterpret_cast<const f32x2*>(row)[p];
  } else {
    const float2 f = halves_of(reinterpret_cast<const uint32_t*>(row)[p], T());
    return pair(f.x, f.y);
  }
}
template <int CH>
__device__ __forceinline__ f32x2& pair_of(float (&row)[CH]) { return reinterpret_cast<f32x2*>(row)[lane_pair<CH>()]; }
// A vector [channels] in 32 bits, zeros where it is NULL or past the tile.
template <int CH>
__device__ __forceinline__ f32x2 channel_pair(const float* v, const ScanTile& t) {
  const int c = 2 * lane_pair<CH>();
  return pair(v && c < t.count ? v[t.first + c] : 0.f, v && c + 1 < t.count ? v[t.first + c + 1] : 0.f);
}
// Writes rows of a tensor by such pairs.
template <class T, int CH>
struct PairOut {
  T* at;
  int64_t stride;
  int count;   // channels of the lane: 0, 1 or 2
  bool whole;  // pairs lie on their own size
  __device__ __forceinline__ PairOut(void* p, int64_t stride, int64_t row, const ScanTile& t)
      : at((T*)p + row * stride + t.first + 2 * lane_pair<CH>()), stride(stride), count(min(t.count - 2 * lane_pair<CH>(), 2)),
        whole((uintptr_t)at % (2 * sizeof(T)) == 0 && stride % 2 == 0) {}
  __device__ __forceinline__ void put(int r, f32x2 v) const {
    const float2 f = halves(v);
    T* to = at + r * stride;
    if (count == 2 && whole) {
      if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(to) = f;
      else *reinterpret_cast<uint32_t*>(to) = word_of(f.x, f.y, T());
    } else {
      if (count > 0) to[0] = RowType<T>::from(f.x);
      if (count > 1) to[1] = RowType<T>::from(f.y);
    }
  }
};
// The steps of a row's channels: dt + bias, or its softplus.
__device__ __forceinline__ f32x2 scan_step_of(f32x2 dt, f32x2 bias, int softplus) {
  const f32x2 v = add2(dt, bias);
  return softplus ? scan_softplus(v) : v;
}
// z sigmoid(z).
__device__ __forceinline__ f32x2 scan_gate(f32x2 z) { return mul2(z, scan_sigmoid(z)); }

// Rows of b or c: kStates states from n0 on, elements 32 apart of kTileRows x kStates.
template <class T, int kStates>
struct ScanStates {
  static constexpr int kEach = kTileRows * kStates / 32, kStep = 32 / kStates;
  const T* from;  // the lane's state of row lane / kStates
  int64_t stride;
  bool is;
  T f[kEach];
  __device__ __forceinline__ ScanStates(const void* src, int64_t stride, int64_t group, int64_t row0, int states, int n0)
      : stride(stride) {
    const int lane = threadIdx.x & 31;
    is = n0 + lane % kStates < states;
    from = (const T*)src + group + n0 + lane % kStates + (row0 + lane / kStates) * stride;
  }
  __device__ __forceinline__ void load(int row, int n) {  // rows [row, row + n) after row0
    const int r = (threadIdx.x & 31) / kStates;
    const T* at = from + row * stride;
#pragma unroll
    for (int i = 0; i < kEach; ++i, at += kStep * stride) f[i] = is && r + i * kStep < n ? *at : RowType<T>::from(0.f);
  }
  __device__ __forceinline__ void store(float (&dst)[kTileRows][kStates]) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kEach; ++i) (&dst[0][0])[lane + 32 * i] = RowType<T>::to(f[i]);
  }
  __device__ __forceinline__ void store(f32x2 (&dst)[kTileRows][kStates]) const {  // twice each
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kEach; ++i) (&dst[0][0])[lane + 32 * i] = both(RowType<T>::to(f[i]));
  }
};

// N pairs that lie on 16 bytes.
template <int N>
__device__ __forceinline__ void read_pairs(f32x2 (&f)[N], const void* at) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const ulonglong2 v = reinterpret_cast<const ulonglong2*>(at)[i / 2];
    f[i] = v.x, f[i + 1] = v.y;
  }
}
__device__ __forceinline__ void write_pairs(void* at, f32x2 x, f32x2 y) { *reinterpret_cast<ulonglong2*>(at) = make_ulonglong2(x, y); }

// N consecutive numbers: in the workspace on 4 N bytes, or on 16; of a dense
// [channels, states] array anywhere.
template <int N>
__device__ __forceinline__ void read_numbers(float (&f)[N], const float* at) {
  if constexpr (N == 2) {
    const float2 v = *reinterpret_cast<const float2*>(at);
    f[0] = v.x, f[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(at + i);
      f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void write_numbers(float* at, const float (&f)[N]) {
  if constexpr (N == 2) {
    *reinterpret_cast<float2*>(at) = make_float2(f[0], f[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(at + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  }
}
// A lane's 4 channels from c4 of the tile, NN states from s, of a dense array;
// zeros where it is NULL or past it.
template <int NN>
__device__ __forceinline__ void read_dense(float (&f)[4][NN], const float* at, const ScanTile& t, int states, int c4, int s) {
  const bool vec = NN % 4 == 0 && states % 4 == 0 && ((uintptr_t)at & 15) == 0 && s + NN <= states;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool is = at && c4 + i < t.count;
    const float* from = at + (int64_t)(t.first + c4 + i) * states + s;
#pragma unroll
    for (int n = 0; n < NN; ++n) f[i][n] = 0.f;
    if (is && vec) {
      read_numbers<NN>(f[i], from);
    } else if (is) {
#pragma unroll
      for (int n = 0; n < NN; ++n)
        if (s + n < states) f[i][n] = from[n];
    }
  }
}
template <int NN>
__device__ __forceinline__ void write_dense(float* at, const float (&f)[4][NN], const ScanTile& t, int states, int c4, int s) {
  const bool vec = NN % 4 == 0 && states % 4 == 0 && ((uintptr_t)at & 15) == 0 && s + NN <= states;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c4 + i < t.count) {
      float* to = at + (int64_t)(t.first + c4 + i) * states + s;
      if (vec) {
        write_numbers<NN>(to, f[i]);
      } else {
#pragma unroll
        for (int n = 0; n < NN; ++n)
          if (s + n < states) to[n] = f[i][n];
      }
    }
}

// Zeros for a tile's channels of the rows that no grid has: a slot's share.
template <class T, int CH>
__device__ __forceinline__ void scan_zero_share(const ScanLaunch& l, void* out, int64_t stride, int slot, const ScanTile& t) {
  const LinCover c = lin_cover(l);
  const int64_t rows = c.begin + l.tokens - c.end;
  if (rows == 0) return;
  const int64_t per = (rows + l.segments - 1) / l.segments, r0 = min(slot * per, rows), r1 = min(r0 + per, rows);
  for (int i = threadIdx.x & 31; i < t.count; i += 32)
    for (int64_t r = r0; r < r1; ++r)
      ((T*)out)[(r < c.begin ? r : r - c.begin + c.end) * stride + t.first + i] = RowType<T>::from(0.f);
}

}  // namespace tb
