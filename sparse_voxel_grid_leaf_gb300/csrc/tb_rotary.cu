// Rotary positions of queries and keys (tb_rotary).
//
// Pair p of a head turns by the angle 2 pi * pos * turns[p].  With turns as
// 64-bit fixed-point fractions of a turn the product's low 64 bits are the
// phase modulo one turn, exactly, for every position; the top 32 bits of it
// are the angle to 2^-32 of a turn, which sincospif takes without a range
// reduction of its own.
//
// Every element is read once and written once, so the bound is memory.  The
// sines and cosines depend on the token and the pair but not on the head: a
// block takes a few tokens, computes their table once into shared memory and
// streams all heads of q and k past it, 16 bytes at a time, four rows of a
// thread in flight.  Measured: 124807 tokens of 8 + 8 heads of 64 in bf16 with
// three position axes 84 us, 6.07 TB/s; the inverse of 20011 tokens of 12 + 4
// heads of 96 in fp32 43 us, 5.71 TB/s; 32 tokens 4.8 us, most of it the launch.
#include "tb_seq.cuh"
#include "tb_seq.h"

namespace tb {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // rows in flight per thread

// A row's units: V pairs that turn -- half layout: elements [V u, V u + V) and
// the same at + pairs; interleaved: 2 V consecutive elements -- and past them
// V elements that pass through.  Pair V u + j of the table is stored at
// [j][u], so that the lanes of a warp read it without bank conflicts.
template <class T, int V, bool kHalf>
__global__ void __launch_bounds__(kThreads) k_rotary(RotaryLaunch r) {
  const tb_rotary_args& a = r.a;
  extern __shared__ float2 s_cs[];  // [per_block, V, pairs / V]
  const int64_t t0 = (int64_t)blockIdx.x * r.per_block;
  const int nt = (int)min((int64_t)r.per_block, a.tokens - t0);
  const int pairs = a.pairs;
  const int turned = pairs / V;                          // units that turn
  const int units = turned + (a.dim - 2 * pairs) / V;    // and that pass through

  const int heads = a.q_heads + a.k_heads;
  const int rows = kThreads / units;
  const int u = threadIdx.x % units, r0 = threadIdx.x / units;
  const bool turn = u < turned;
  // element offsets of the unit's one or two vectors
  const int e0 = turn ? (kHalf ? u * V : 2 * u * V) : 2 * pairs + (u - turned) * V;
  const int e1 = kHalf ? e0 + pairs : e0 + V;
  const int step_t = rows / heads, step_h = rows - step_t * heads;
  int t = r0 / heads, h = r0 - t * heads;
  if (r0 >= rows) t = nt;  // threads past the last whole row

  Pack<T, V> x[kBatch], y[kBatch];
  T* dst[kBatch];
  int tok[kBatch];
  auto load = [&] {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      tok[i] = t;
      if (t < nt) {
        const bool isq = h < a.q_heads;
        const int hh = isq ? h : h - a.q_heads;
        const T* src = (const T*)(isq ? a.q : a.k) + (t0 + t) * (isq ? a.q_row : a.k_row) +
                       hh * (isq ? a.q_head : a.k_head);
        dst[i] = (T*)(isq ? a.q_out : a.k_out) + (t0 + t) * (isq ? a.q_out_row : a.k_out_row) +
                 hh * (isq ? a.q_out_head : a.k_out_head);
        x[i] = load_pack<T, V>(src + e0);
        if (turn) y[i] = load_pack<T, V>(src + e1);
      }
      t += step_t;
      h += step_h;
      if (h >= heads) {
        h -= heads;
        ++t;
      }
    }
  };
  load();  // on their way while the table is made

  const float sign = a.inverse ? -a.amplitude : a.amplitude;
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, p = i - t * pairs;
    int axis = 0;
    if (a.axes > 1) {
      const int s1 = a.section[0], s2 = s1 + a.section[1];
      axis = p < s1 ? 0 : (p < s2 || a.axes == 2) ? 1 : 2;
    }
    const int64_t at = (t0 + t) * a.position_row + axis;
    const int64_t pos = a.positions64 ? ((const int64_t*)a.positions)[at] : (int64_t)((const int32_t*)a.positions)[at];
    const uint64_t phase = (uint64_t)pos * (uint64_t)a.turns[p];
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
    s_cs[t * pairs + p % V * turned + p / V] = make_float2(c * a.amplitude, s * sign);
  }
  __syncthreads();

  while (tok[0] < nt) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (tok[i] >= nt) break;
      if (turn) {
        float fx[V], fy[V];
        unpack<T, V>(x[i], fx);
        unpack<T, V>(y[i], fy);
        const float2* cs = s_cs + tok[i] * pairs + u;
        if constexpr (kHalf || V == 1) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float2 w = cs[j * turned];
            const float p = fx[j] * w.x - fy[j] * w.y, q = fy[j] * w.x + fx[j] * w.y;
            fx[j] = p;
            fy[j] = q;
          }
        } else {
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            const float2 w = cs[j / 2 * turned], z = cs[(V + j) / 2 * turned];
            float p = fx[j] * w.x - fx[j + 1] * w.y, q = fx[j + 1] * w.x + fx[j] * w.y;
            fx[j] = p;
            fx[j + 1] = q;
            p = fy[j] * z.x - fy[j + 1] * z.y;
            q = fy[j + 1] * z.x + fy[j] * z.y;
            fy[j] = p;
            fy[j + 1] = q;
          }
        }
        store_pack<T, V>(dst[i] + e0, pack<T, V>(fx));
        store_pack<T, V>(dst[i] + e1, pack<T, V>(fy));
      } else {
        store_pack<T, V>(dst[i] + e0, x[i]);
      }
    }
    load();
  }
}

template <class T, int V>
cudaError_t go(const RotaryLaunch& r, cudaStream_t s) {
  const int64_t blocks = (r.a.tokens + r.per_block - 1) / r.per_block;
  const size_t smem = (size_t)r.per_block * r.a.pairs * sizeof(float2);
  if (r.a.layout == 0) k_rotary<T, V, true><<<(unsigned)blocks, kThreads, smem, s>>>(r);
  else k_rotary<T, V, false><<<(unsigned)blocks, kThreads, smem, s>>>(r);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const void* args, cudaStream_t s) {
  const RotaryLaunch& r = *(const RotaryLaunch*)args;
  switch (r.a.type) {
    case TB_TYPE_F32: return r.vec == 4 ? go<float, 4>(r, s) : go<float, 1>(r, s);
    case TB_TYPE_F16: return r.vec == 8 ? go<__half, 8>(r, s) : r.vec == 4 ? go<__half, 4>(r, s) : go<__half, 1>(r, s);
    default:
      return r.vec == 8 ? go<__nv_bfloat16, 8>(r, s)
             : r.vec == 4 ? go<__nv_bfloat16, 4>(r, s) : go<__nv_bfloat16, 1>(r, s);
  }
}

}  // namespace tb
