// What the kernels of the selective scan share: how a warp's lanes hold a tile
// of channels and states, rows through shared memory, the functions of a step.
//
// A warp walks down the rows of a tile of 32 channels (kScanChannels) and 4 NN
// states.  Lane l holds channels 4 (l / 4) .. + 4 and states NN (l % 4) .. + NN
// of it, 4 NN numbers, so that a row costs it one 16-byte read each of delta
// and delta x (of its channels) and one or two of b and c (of its states) for 4
// NN updates of h; a sum over the states is one over its own and 4 lanes, a sum
// over the channels one over its own and 8 lanes.  Both go through shared
// memory: a lane writes its own sums, and the lane of a channel (or state)
// reads and adds what belongs to it.
#pragma once

#include "tb_linattn.cuh"
#include "tb_seq.cuh"

namespace tb {

constexpr int kScanRows = 8;  // of a tile in shared memory
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float scan_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(delta a) for a2 = a log2(e).  The instruction rounds towards zero: over
// [-1, 0] its results are 2e-8 to 5e-8 low on average (measured), which the
// many decays that a slow state goes through would add up.  2^-25 more in the
// exponent takes most of that back, and costs nothing as a sum.
__device__ __forceinline__ float scan_decay(float delta, float a2) { return scan_ex2(fmaf(delta, a2, 0x1p-25f)); }

// log(1 + exp(v)) = max(v, 0) + log(1 + u), u = exp(-|v|), and log(1 + u) = 2
// artanh(s), s = u / (2 + u) <= 1/3, by its series: small steps keep their
// relative accuracy.  exp(-|v|) gets the rest of the product with log2(e) back.
__device__ __forceinline__ float scan_softplus(float v) {
  const float m = -fabsf(v), e = m * kLog2e;
  const float rest = fmaf(m, kLog2e, -e) + m * 1.9259629e-8f;  // log2(e) in 32 bits is short of this
  float u = scan_ex2(e);
  u = fmaf(u, rest * kLn2, u);
  if (v != v || e < -1e30f) u = scan_ex2(e);  // infinite: the rest is no number
  const float s = __fdividef(u, 2.f + u), q = s * s;
  float p = 1.f / 13.f;
  p = fmaf(p, q, 1.f / 11.f);
  p = fmaf(p, q, 1.f / 9.f);
  p = fmaf(p, q, 1.f / 7.f);
  p = fmaf(p, q, 1.f / 5.f);
  p = fmaf(p, q, 1.f / 3.f);
  return fmaxf(v, 0.f) + 2.f * fmaf(s * q, p, s);
}
__device__ __forceinline__ float scan_sigmoid(float v) { return __fdividef(1.f, 1.f + scan_ex2(-v * kLog2e)); }

__device__ __forceinline__ void copy_row(void* dst, const void* src, int bytes) {  // 16 bytes, zeros past `bytes`
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(bytes)
               : "memory");
}

// The channels of a warp.
struct ScanTile {
  int group, first, count;  // first channel of all; count <= 0: none
};
__device__ __forceinline__ ScanTile scan_tile(const ScanLaunch& l, int group, int tile) {
  const int per = l.a.channels / l.a.groups;
  return {group, group * per + tile * kScanChannels, tile < l.group_tiles ? min(kScanChannels, per - tile * kScanChannels) : 0};
}

// Rows [row, row + n) of a tile's channels to dst [kScanRows][kScanChannels],
// zeros past them; asynchronous where vectors fit.
template <class T>
__device__ __forceinline__ void scan_fetch(T* dst, const void* src, int64_t stride, int64_t row, int n, const ScanTile& t, bool vec) {
  const int lane = threadIdx.x & 31;
  const T* from = (const T*)src + t.first;
  if (vec && t.count == kScanChannels) {
    constexpr int kChunk = 16 / (int)sizeof(T), kPer = kScanChannels / kChunk;
#pragma unroll
    for (int i = lane; i < kScanRows * kPer; i += 32) {
      const int r = i / kPer, c = i % kPer * kChunk;
      copy_row(dst + r * kScanChannels + c, from + (row + min(r, max(n - 1, 0))) * stride + c, r < n ? 16 : 0);
    }
  } else {
#pragma unroll
    for (int r = 0; r < kScanRows; ++r)
      dst[r * kScanChannels + lane] = r < n && lane < t.count ? from[(row + r) * stride + lane] : RowType<T>::from(0.f);
  }
}
__device__ __forceinline__ void scan_fetched() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void scan_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  __syncwarp();
}

// Rows of b or c: 4 NN states from n0 on, elements 32 apart of kScanRows x 4 NN.
template <class T, int NN>
struct ScanStates {
  static constexpr int kStates = 4 * NN, kEach = kScanRows * kStates / 32;
  float f[kEach];
  __device__ __forceinline__ void load(const void* src, int64_t stride, int64_t group, int64_t row, int n, int states, int n0) {
    const int lane = threadIdx.x & 31, s = lane % kStates;
    const T* from = (const T*)src + group + n0 + s;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int r = lane / kStates + i * (32 / kStates);
      f[i] = r < n && n0 + s < states ? RowType<T>::to(from[(row + r) * stride]) : 0.f;
    }
  }
  __device__ __forceinline__ void store(float* dst) const {  // [kScanRows][kStates]
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kEach; ++i) dst[lane + 32 * i] = f[i];
  }
};

template <int NN>
__device__ __forceinline__ void read_states(float (&f)[NN], const float* at) {
  if constexpr (NN == 4) {
    const float4 v = *reinterpret_cast<const float4*>(at);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(at);
    f[0] = v.x, f[1] = v.y;
  }
}
__device__ __forceinline__ void read_channels(float (&f)[4], const float* at) { read_states<4>(f, at); }
__device__ __forceinline__ void write_channels(float* at, const float (&f)[4]) {
  *reinterpret_cast<float4*>(at) = make_float4(f[0], f[1], f[2], f[3]);
}

// A lane's numbers of a [.., channels, pad] array of the workspace: 16 or 8
// bytes for each of its channels.
template <int NN>
__device__ __forceinline__ void read_pad(float (&h)[4][NN], const float* at, const ScanTile& t, int pad, int n0) {
  const int lane = threadIdx.x & 31, c = lane / 4 * 4, s = n0 + lane % 4 * NN;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (c + i < t.count) read_states<NN>(h[i], at + (int64_t)(t.first + c + i) * pad + s);
    else
#pragma unroll
      for (int n = 0; n < NN; ++n) h[i][n] = 0.f;
  }
}
template <int NN>
__device__ __forceinline__ void write_pad(float* at, const float (&h)[4][NN], const ScanTile& t, int pad, int n0) {
  const int lane = threadIdx.x & 31, c = lane / 4 * 4, s = n0 + lane % 4 * NN;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c + i < t.count) {
      float* to = at + (int64_t)(t.first + c + i) * pad + s;
      if constexpr (NN == 4) *reinterpret_cast<float4*>(to) = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
      else *reinterpret_cast<float2*>(to) = make_float2(h[i][0], h[i][1]);
    }
}
// The same of a [channels, states] array, element by element (a is one of them).
template <int NN>
__device__ __forceinline__ void read_dense(float (&h)[4][NN], const float* at, const ScanTile& t, int states, int n0) {
  const int lane = threadIdx.x & 31, c = lane / 4 * 4, s = n0 + lane % 4 * NN;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int n = 0; n < NN; ++n)
      h[i][n] = at && c + i < t.count && s + n < states ? at[(int64_t)(t.first + c + i) * states + s + n] : 0.f;
}
template <int NN>
__device__ __forceinline__ void write_dense(float* at, const float (&h)[4][NN], const ScanTile& t, int states, int n0) {
  const int lane = threadIdx.x & 31, c = lane / 4 * 4, s = n0 + lane % 4 * NN;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int n = 0; n < NN; ++n)
      if (c + i < t.count && s + n < states) at[(int64_t)(t.first + c + i) * states + s + n] = h[i][n];
}

// Zeros for a tile's channels of the rows that no grid has: a slot's share.
template <class T>
__device__ __forceinline__ void scan_zero_share(const ScanLaunch& l, void* out, int64_t stride, int slot, const ScanTile& t) {
  const LinCover c = lin_cover(l);
  const int64_t rows = c.begin + l.tokens - c.end;
  if (rows == 0) return;
  const int64_t per = (rows + l.segments - 1) / l.segments, r0 = min(slot * per, rows), r1 = min(r0 + per, rows);
  const int lane = threadIdx.x & 31;
  if (lane < t.count)
    for (int64_t r = r0; r < r1; ++r)
      ((T*)out)[(r < c.begin ? r : r - c.begin + c.end) * stride + t.first + lane] = RowType<T>::from(0.f);
}

}  // namespace tb
