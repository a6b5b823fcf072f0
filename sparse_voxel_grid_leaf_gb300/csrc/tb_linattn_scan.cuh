// The recurrence over the rows of one segment and head, in 32-bit arithmetic:
// any row type, head size and decay.
//
// A warp holds the state columns of 16 values, each thread 2 columns x a
// quarter of the keys in registers, and walks the rows, which the block stages
// in shared memory as floats.  Two multiply-adds and a multiply per state
// element and row, in packed pairs (fma.rn.f32x2), bound it where walks are
// many (512 grids of 8 rows, 8 heads of 128 x 128: 98 us), the loads of 16 rows
// and their turn through shared memory where they are few (a token of 7 heads
// 4.2 us; 30 grids of 6 or 7 rows, 8 heads of 128 x 64: 8.3 us).
#pragma once

#include "tb_linattn.cuh"
#include "tb_seq.cuh"

namespace tb {

typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

constexpr int kScanRows = 16;  // rows staged at a time
constexpr int scan_floats(int KS) { return kScanRows * (2 * 4 * KS + 128); }

// By the block's first `threads` threads (whole warps, 16 values each), which
// alone meet at barrier 1.  KS: keys of one thread; 4 KS >= K.  A warp's four
// key slices interleave by four keys, so that their 16-byte reads of a staged
// row are consecutive.  s_rows: scan_floats(KS) floats, 16-byte aligned.
template <class T, int KS>
__device__ __forceinline__ void scan_walk(const LinLaunch& l, const LinProblem& p, const LinSegment& seg, int h,
                                          float* s_rows, int threads) {
  constexpr int KP = 4 * KS;
  float(*s_a)[KP] = reinterpret_cast<float(*)[KP]>(s_rows);
  float(*s_b)[KP] = s_a + kScanRows;
  float(*s_c)[128] = reinterpret_cast<float(*)[128]>(s_b + kScanRows);
  const bool want_out = p.out && l.phase != 1;
  if (l.phase == 1 && seg.index + 1 == seg.count && !p.last) return;  // nobody reads this segment's state
  const float decay = l.decay[h];
  const int lane = threadIdx.x & 31, slice = lane & 3, warp = threadIdx.x >> 5, warps = threads >> 5;
  const T zero = RowType<T>::from(0.f);
  const int v0 = (threadIdx.x >> 5) * 16 + (lane >> 2) * 2;
  const int64_t state_at = ((int64_t)seg.grid * l.heads + h) * p.K * p.V;
  float* seg_state = p.seg ? p.seg + ((int64_t)seg.slot * l.heads + h) * p.K * p.V : nullptr;

  f32x2 u[2][KS / 2] = {};
  auto key = [&](int i) { return (i / 4 * 4 + slice) * 4 + i % 4; };
  const float* from = l.phase == 2 ? seg_state : l.phase == 0 && p.first ? p.first + state_at : nullptr;
  if (from) {
    const int64_t by_k = l.phase == 2 ? p.V : p.first_k, by_v = l.phase == 2 ? 1 : p.first_v;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < KS; i += 2) {
        float x[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          x[j] = key(i + j) < p.K && v0 + c < p.V ? from[key(i + j) * by_k + (v0 + c) * by_v] : 0.f;
        u[c][i / 2] = pair(x[0], x[1]);
      }
  }

  const int64_t origin = p.reverse ? seg.end - 1 - seg.first : seg.begin + seg.first;
  const int64_t dir = p.reverse ? -1 : 1;
  const f32x2 fold = pair(p.fold, p.fold);
#pragma unroll 1
  for (int t0 = 0; t0 < seg.len; t0 += kScanRows) {
    const int nt = min(kScanRows, seg.len - t0);
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
    // two rows of a warp in flight
    for (int t = 2 * warp; t < nt; t += 2 * warps) {
      T x[2][KP / 32], y[2][KP / 32], z[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t row = origin + dir * (t0 + t + r);
        const T* a = (const T*)p.a + row * p.a_row + h * p.a_head;
        const T* b = (const T*)p.b + row * p.b_row + h * p.b_head;
        const T* c = (const T*)p.c + row * p.c_row + h * p.c_head;
        const bool live = t + r < nt;
#pragma unroll
        for (int i = 0; i < KP / 32; ++i) {
          const int k = i * 32 + lane;
          x[r][i] = live && want_out && k < p.K ? a[k] : zero;
          y[r][i] = live && k < p.K ? b[k] : zero;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) z[r][i] = live && i * 32 + lane < p.V ? c[i * 32 + lane] : zero;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int i = 0; i < KP / 32; ++i) {
          s_a[t + r][i * 32 + lane] = RowType<T>::to(x[r][i]);
          s_b[t + r][i * 32 + lane] = RowType<T>::to(y[r][i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s_c[t + r][i * 32 + lane] = RowType<T>::to(z[r][i]);
      }
    }
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
      const float d = p.late && t0 + t == 0 ? 1.f : decay;
      const f32x2 d2 = pair(d, d);
      const f32x2 c0 = mul2(pair(s_c[t][v0], s_c[t][v0]), fold);
      const f32x2 c1 = mul2(pair(s_c[t][v0 + 1], s_c[t][v0 + 1]), fold);
      f32x2 o0 = 0ull, o1 = 0ull;
#pragma unroll
      for (int i = 0; i < KS; i += 4) {
        const float4 b = *reinterpret_cast<const float4*>(&s_b[t][(i + slice) * 4]);
        const f32x2 b0 = pair(b.x, b.y), b1 = pair(b.z, b.w);
        u[0][i / 2] = fma2(u[0][i / 2], d2, mul2(b0, c0));
        u[1][i / 2] = fma2(u[1][i / 2], d2, mul2(b0, c1));
        u[0][i / 2 + 1] = fma2(u[0][i / 2 + 1], d2, mul2(b1, c0));
        u[1][i / 2 + 1] = fma2(u[1][i / 2 + 1], d2, mul2(b1, c1));
        if (want_out) {
          const float4 a = *reinterpret_cast<const float4*>(&s_a[t][(i + slice) * 4]);
          const f32x2 a0 = pair(a.x, a.y), a1 = pair(a.z, a.w);
          o0 = fma2(a0, u[0][i / 2], o0);
          o1 = fma2(a0, u[1][i / 2], o1);
          o0 = fma2(a1, u[0][i / 2 + 1], o0);
          o1 = fma2(a1, u[1][i / 2 + 1], o1);
        }
      }
      if (want_out) {
        float x = halves(o0).x + halves(o0).y, y = halves(o1).x + halves(o1).y;
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        y += __shfl_xor_sync(0xffffffffu, y, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        y += __shfl_xor_sync(0xffffffffu, y, 2);
        const int v = v0 + slice;
        if (slice < 2 && v < p.V) {
          const int64_t row = origin + dir * (t0 + t);
          ((T*)p.out)[row * p.o_row + h * p.o_head + v] = RowType<T>::from((slice ? y : x) * p.mul);
        }
      }
    }
  }

  float* dst = l.phase == 1 ? seg_state : l.phase == 0 && p.last ? p.last + state_at : nullptr;
  if (!dst) return;
  const float leave = p.late && seg.len > 0 ? decay : 1.f;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < KS; i += 2) {
      const float2 x = halves(u[c][i / 2]);
      const int v = v0 + c;
      if (v < p.V && key(i) < p.K) dst[(int64_t)key(i) * p.V + v] = x.x * leave;
      if (v < p.V && key(i + 1) < p.K) dst[(int64_t)key(i + 1) * p.V + v] = x.y * leave;
    }
}

}  // namespace tb
