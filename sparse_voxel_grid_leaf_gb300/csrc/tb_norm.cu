// Root-mean-square norm with the residual stream's addition, an output in
// e4m3 with a scale for each row, and the gradient (tb_rms_norm,
// tb_rms_norm_backward).
//
// All bytes are read once and written once, so the bound is memory: a row's
// elements stay in the registers of its threads between the sum of squares
// and the output (per_row threads of nv vectors each; rows narrower than
// a block share it).
#include "tb_seq.cuh"
#include "tb_seq.h"

namespace tb {
namespace {

constexpr int kMaxThreads = 512;

// Sum (or maximum) of one value over the threads of a row: threadIdx.x runs
// over the row, warps are whole.  Rows of one warp need no barrier.
template <bool kMax>
__device__ __forceinline__ float row_reduce(float x, float* s, int& turn) {
  x = kMax ? warp_max(x) : warp_sum(x);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return x;
  float* at = s + (turn ^= 1) * 32;
  if ((threadIdx.x & 31) == 0) at[threadIdx.y * warps + (threadIdx.x >> 5)] = x;
  __syncthreads();
  float v = at[threadIdx.y * warps];
  for (int i = 1; i < warps; ++i) v = kMax ? fmaxf(v, at[threadIdx.y * warps + i]) : v + at[threadIdx.y * warps + i];
  return v;
}

template <class T, int V, int NV, bool kFp8>
__global__ void __launch_bounds__(kMaxThreads) k_norm(NormLaunch n) {
  const tb_norm_args& a = n.a;
  __shared__ float s_red[64];
  int turn = 0;
  const int vecs = a.width / V;
  const float inv_width = 1.f / (float)a.width;
  const T* w = (const T*)a.weight;
  // block-uniform trip count: the barriers of row_reduce are passed by all
  for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < a.rows; base += (int64_t)gridDim.x * blockDim.y) {
    const int64_t row = base + threadIdx.y;
    const bool live = row < a.rows;
    float f[NV][V];
    const T* x = (const T*)a.x + row * a.x_row;
    const T* res = (const T*)a.residual + row * a.residual_row;
    float sum = 0.f;
    {
      Pack<T, V> px[NV], pr[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (live && v < vecs) {
          px[i] = load_pack<T, V>(x + (int64_t)v * V);
          if (a.residual) pr[i] = load_pack<T, V>(res + (int64_t)v * V);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (live && v < vecs) {
          unpack<T, V>(px[i], f[i]);
          if (a.residual) {
            float g[V];
            unpack<T, V>(pr[i], g);
#pragma unroll
            for (int j = 0; j < V; ++j) f[i][j] += g[j];
            if (a.h_out) store_pack<T, V>((T*)a.h_out + row * a.h_row + (int64_t)v * V, pack<T, V>(f[i]));
          }
#pragma unroll
          for (int j = 0; j < V; ++j) sum = fmaf(f[i][j], f[i][j], sum);
        }
      }
    }
    sum = row_reduce<false>(sum, s_red, turn);
    const float r = rsqrtf(fmaf(sum, inv_width, a.eps));
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (live && v < vecs) {
        float g[V];
        unpack<T, V>(load_pack<T, V>(w + (int64_t)v * V), g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          f[i][j] *= r * g[j];
          if (kFp8) top = fmaxf(top, fabsf(f[i][j]));
        }
        if constexpr (!kFp8)
          store_pack<T, V>((T*)a.y + row * a.y_row + (int64_t)v * V, pack<T, V>(f[i]));
      }
    }
    if constexpr (kFp8) {
      // A NaN in a row makes all of its y NaN; fmaxf drops them (scale 0) and
      // the conversion keeps them.
      top = row_reduce<true>(top, s_red, turn);
      const float scale = top * (1.f / 448.f);
      const float inv = top > 0.f ? 448.f / top : 0.f;
      if (live && threadIdx.x == 0) a.scale[row] = scale;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (live && v < vecs) {
          uint8_t* dst = (uint8_t*)a.y + row * a.y_row + (int64_t)v * V;
          if constexpr (V == 1) {
            *dst = __nv_cvt_float_to_fp8(f[i][0] * inv, __NV_SATFINITE, __NV_E4M3);
          } else {
            uint32_t word[V / 4];
#pragma unroll
            for (int j = 0; j < V; j += 4) {
              const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[i][j] * inv, f[i][j + 1] * inv),
                                                           __NV_SATFINITE, __NV_E4M3);
              const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[i][j + 2] * inv, f[i][j + 3] * inv),
                                                           __NV_SATFINITE, __NV_E4M3);
              word[j / 4] = lo | hi << 16;
            }
            if constexpr (V == 8) *(uint2*)dst = make_uint2(word[0], word[1]);
            else *(uint32_t*)dst = word[0];
          }
        }
      }
    }
  }
}

// Rows of dx, and a block's part of dweight in registers over its rows: part
// [blocks, width] in the workspace, summed by k_norm_weight in a fixed order.
template <class T, int V, int NV>
__global__ void __launch_bounds__(kMaxThreads) k_norm_backward(NormBackwardLaunch n) {
  const tb_norm_backward_args& a = n.a;
  extern __shared__ float s_part[];  // [rows, per_row * NV * V] where a block has more than one row
  __shared__ float s_red[64];
  int turn = 0;
  const int vecs = a.width / V;
  const float inv_width = 1.f / (float)a.width;
  float dw[NV][V] = {};
  for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < a.rows; base += (int64_t)gridDim.x * blockDim.y) {
    const int64_t row = base + threadIdx.y;
    const bool live = row < a.rows;
    Pack<T, V> ph[NV], pd[NV], pg[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (live && v < vecs) {
        ph[i] = load_pack<T, V>((const T*)a.h + row * a.h_row + (int64_t)v * V);
        pd[i] = load_pack<T, V>((const T*)a.dy + row * a.dy_row + (int64_t)v * V);
        if (a.dh) pg[i] = load_pack<T, V>((const T*)a.dh + row * a.dh_row + (int64_t)v * V);
      }
    }
    float hh = 0.f, hd = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (live && v < vecs) {
        float h[V], d[V], w[V];
        unpack<T, V>(ph[i], h);
        unpack<T, V>(pd[i], d);
        unpack<T, V>(load_pack<T, V>((const T*)a.weight + (int64_t)v * V), w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          hh = fmaf(h[j], h[j], hh);
          hd = fmaf(h[j] * w[j], d[j], hd);
        }
      }
    }
    hh = row_reduce<false>(hh, s_red, turn);
    hd = row_reduce<false>(hd, s_red, turn);
    const float r = rsqrtf(fmaf(hh, inv_width, a.eps));
    const float m = r * r * r * hd * inv_width;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (live && v < vecs) {
        float h[V], d[V], w[V], g[V];
        unpack<T, V>(ph[i], h);
        unpack<T, V>(pd[i], d);
        unpack<T, V>(load_pack<T, V>((const T*)a.weight + (int64_t)v * V), w);
        if (a.dh) unpack<T, V>(pg[i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          dw[i][j] = fmaf(d[j], h[j] * r, dw[i][j]);
          const float x = fmaf(-m, h[j], r * w[j] * d[j]);
          h[j] = a.dh ? x + g[j] : x;
        }
        store_pack<T, V>((T*)a.dx + row * a.dx_row + (int64_t)v * V, pack<T, V>(h));
      }
    }
  }
  float* part = a.workspace + (int64_t)blockIdx.x * a.width;
  if (blockDim.y > 1) {
    const int span = blockDim.x * NV * V;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) s_part[threadIdx.y * span + (i * V + j) * blockDim.x + threadIdx.x] = dw[i][j];
    __syncthreads();
    if (threadIdx.y == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
          for (int y = 1; y < blockDim.y; ++y) dw[i][j] += s_part[y * span + (i * V + j) * blockDim.x + threadIdx.x];
    }
  }
  if (threadIdx.y == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vecs)
#pragma unroll
        for (int j = 0; j < V; ++j) part[v * V + j] = dw[i][j];
    }
  }
}

// dweight = the blocks' parts summed: 32 columns a block, 32 groups of parts.
template <class T>
__global__ void __launch_bounds__(1024) k_norm_weight(NormBackwardLaunch n) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float sum = 0.f;
  if (c < n.a.width)
    for (int b = threadIdx.y; b < n.blocks; b += 32) sum += n.a.workspace[(int64_t)b * n.a.width + c];
  s[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  const float all = warp_sum(s[threadIdx.x][threadIdx.y]);
  const int o = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && o < n.a.width) ((T*)n.a.dweight)[o] = RowType<T>::from(all);
}

template <class T, int V, int NV>
cudaError_t go(const NormLaunch& n, cudaStream_t s) {
  const dim3 block(n.per_row, n.rows);
  if (n.a.fp8) k_norm<T, V, NV, true><<<n.blocks, block, 0, s>>>(n);
  else k_norm<T, V, NV, false><<<n.blocks, block, 0, s>>>(n);
  return cudaGetLastError();
}

template <class T>
cudaError_t pick(const NormLaunch& n, cudaStream_t s) {
  constexpr int V = RowType<T>::kVec;
  if (n.vec) {
    switch (n.nv) {
      case 1: return go<T, V, 1>(n, s);
      case 2: return go<T, V, 2>(n, s);
      case 4: return go<T, V, 4>(n, s);
      default: return go<T, V, 8>(n, s);
    }
  }
  return n.nv <= 8 ? go<T, 1, 8>(n, s) : go<T, 1, 32>(n, s);
}

template <class T, int V, int NV>
cudaError_t go_back(const NormBackwardLaunch& n, cudaStream_t s) {
  const dim3 block(n.per_row, n.rows);
  const size_t smem = n.rows > 1 ? sizeof(float) * n.rows * n.per_row * NV * V : 0;
  k_norm_backward<T, V, NV><<<n.blocks, block, smem, s>>>(n);
  return cudaGetLastError();
}

template <class T>
cudaError_t pick_back(const NormBackwardLaunch& n, cudaStream_t s) {
  constexpr int V = RowType<T>::kVec;
  if (n.vec) {
    switch (n.nv) {
      case 1: return go_back<T, V, 1>(n, s);
      case 2: return go_back<T, V, 2>(n, s);
      case 4: return go_back<T, V, 4>(n, s);
      default: return go_back<T, V, 8>(n, s);
    }
  }
  return n.nv <= 8 ? go_back<T, 1, 8>(n, s) : go_back<T, 1, 32>(n, s);
}

}  // namespace

cudaError_t launch_norm(const void* args, cudaStream_t s) {
  const NormLaunch& n = *(const NormLaunch*)args;
  switch (n.a.type) {
    case TB_TYPE_F32: return pick<float>(n, s);
    case TB_TYPE_F16: return pick<__half>(n, s);
    default: return pick<__nv_bfloat16>(n, s);
  }
}

cudaError_t launch_norm_backward(const void* args, cudaStream_t s) {
  const NormBackwardLaunch& n = *(const NormBackwardLaunch*)args;
  switch (n.a.type) {
    case TB_TYPE_F32: return pick_back<float>(n, s);
    case TB_TYPE_F16: return pick_back<__half>(n, s);
    default: return pick_back<__nv_bfloat16>(n, s);
  }
}

cudaError_t launch_norm_weight(const void* args, cudaStream_t s) {
  const NormBackwardLaunch& n = *(const NormBackwardLaunch*)args;
  const dim3 block(32, 32);
  const int blocks = (n.a.width + 31) / 32;
  switch (n.a.type) {
    case TB_TYPE_F32: k_norm_weight<float><<<blocks, block, 0, s>>>(n); break;
    case TB_TYPE_F16: k_norm_weight<__half><<<blocks, block, 0, s>>>(n); break;
    default: k_norm_weight<__nv_bfloat16><<<blocks, block, 0, s>>>(n); break;
  }
  return cudaGetLastError();
}

}  // namespace tb
