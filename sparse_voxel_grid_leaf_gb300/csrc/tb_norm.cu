// Root-mean-square norm with the residual stream's addition, an output in
// e4m3 with a scale for each row, and the gradient (tb_rms_norm,
// tb_rms_norm_backward).
//
// All bytes are read once and written once, so the bound is memory: a row's
// elements stay in the registers of its threads between the sum of squares
// and the output (per_row threads of nv vectors each; rows narrower than
// a block share it).  The gradient adds two sums of a row and holds a part of
// dweight in registers as well; its blocks' parts, a few MB, are joined by a
// second kernel.  Measured, bf16: 124807 rows of 1024 with the residual's
// addition 155 us, 6.58 TB/s; the gradient of 60013 rows of 1536 133 us, 5.5
// TB/s (its instructions take 73% of the issue slots, as the forward's do);
// 16 rows of 2048 to e4m3 5.5 us, most of it the launch.
#include "tb_seq.cuh"
#include "tb_seq.h"

namespace tb {
namespace {

constexpr int kMaxThreads = 512;
__host__ __device__ constexpr int up_to(int x, int m) { return (x + m - 1) / m * m; }

// Sums (the second one: sum or maximum) of two values over the threads of a
// row: threadIdx.x runs over the row, which has whole warps, or 4, 8 or 16
// lanes of one.  Rows of one warp or less need no barrier.
template <bool kMax>
__device__ __forceinline__ float2 row_reduce(float x, float y, float2* s, int& turn) {
  const int warps = blockDim.x >> 5;
  if (!warps) {
    for (int o = blockDim.x >> 1; o; o >>= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      const float z = __shfl_xor_sync(0xffffffffu, y, o);
      y = kMax ? fmaxf(y, z) : y + z;
    }
    return make_float2(x, y);
  }
  x = warp_sum(x);
  y = kMax ? warp_max(y) : warp_sum(y);
  if (warps == 1) return make_float2(x, y);
  float2* at = s + (turn ^= 1) * 32;
  if ((threadIdx.x & 31) == 0) at[threadIdx.y * warps + (threadIdx.x >> 5)] = make_float2(x, y);
  __syncthreads();
  float2 v = at[threadIdx.y * warps];
  for (int i = 1; i < warps; ++i) {
    const float2 w = at[threadIdx.y * warps + i];
    v.x += w.x;
    v.y = kMax ? fmaxf(v.y, w.y) : v.y + w.y;
  }
  return v;
}

// Whether a thread has registers for the next row and the weight next to its
// row (30000 rows of 4096 in 16 bits, four vectors a thread: 89 us so, 113 with
// the loads at the row; of 8192, eight vectors: 492 and 181).  The gradient
// holds dweight as well (15000 rows of 16384, four vectors: 869 and 367).
template <class T, int V, int NV, bool kBackward>
constexpr bool ahead() {
  return NV * (V * (int)sizeof(T) + 3) / 4 <= (kBackward ? 16 : 32);
}

// What takes a row's h w to e4m3, from top = max |h w| and r: max |y| is r top,
// and y / scale is h w 448 / top.  448 / top is beyond 32 bits for a top below
// 2^-119, so h w of rows below 2^-100 is raised by 2^100, exactly, before the
// quotient meets it; and h meets w first, as a large weight may stand at a zero.
// A NaN in a row makes all of its y NaN; fmaxf drops them (scale 0 or finite)
// and the conversion keeps them.
struct Fp8Row {
  float scale, up, by;
  __device__ __forceinline__ float operator()(float h, float w) const { return h * w * up * by; }
};
__device__ __forceinline__ Fp8Row fp8_row(float top, float r) {
  const float most = top * r, up = top < 0x1p-100f ? 0x1p100f : 1.f;
  return {most > 0.f ? most * (1.f / 448.f) : 0.f, up, most > 0.f ? 448.f / (top * up) : most == 0.f ? 0.f : r};
}

// Blocks stay and walk over rows; a row's elements are loaded while the one
// before it is normed, and held as they came (16-bit pairs): the sum of the
// residual stream is computed once for the mean and once for the output.
template <class T, int V, int NV, bool kFp8>
__global__ void __launch_bounds__(kMaxThreads) k_norm(NormLaunch n) {
  const tb_norm_args& a = n.a;
  __shared__ float2 s_red[64];
  int turn = 0;
  const int vecs = a.width / V;
  const float inv_width = 1.f / (float)a.width;
  const int64_t stride = (int64_t)gridDim.x * blockDim.y;
  constexpr bool kAhead = ahead<T, V, NV, false>();
  Pack<T, V> w[NV], px[NV], pr[NV];
  auto load = [&](int64_t row) {
    const T* x = (const T*)a.x + row * a.x_row;
    const T* res = (const T*)a.residual + row * a.residual_row;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (row < a.rows && v < vecs) {
        px[i] = load_pack<T, V>(x + (int64_t)v * V);
        if (a.residual) pr[i] = load_pack<T, V>(res + (int64_t)v * V);
      }
    }
  };
  int64_t base = (int64_t)blockIdx.x * blockDim.y;
  if (kAhead) load(base + threadIdx.y);
  auto weight = [&](int i) { return load_pack<T, V>((const T*)a.weight + (int64_t)(threadIdx.x + i * blockDim.x) * V); };
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (kAhead && threadIdx.x + i * blockDim.x < vecs) w[i] = weight(i);
  // block-uniform trip count: the barriers of row_reduce are passed by all
  for (; base < a.rows; base += stride) {
    const int64_t row = base + threadIdx.y;
    const bool live = row < a.rows;
    Pack<T, V> cx[NV], cr[NV];
    if (!kAhead) load(row);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cx[i] = px[i];
      cr[i] = pr[i];
    }
    if (kAhead) load(row + stride);
    auto sum_of = [&](int i, float (&f)[V]) {
      unpack<T, V>(cx[i], f);
      if (a.residual) {
        float g[V];
        unpack<T, V>(cr[i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] += g[j];
      }
    };
    float sum = 0.f, top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (live && v < vecs) {
        float f[V];
        sum_of(i, f);
        if (a.h_out) store_pack<T, V>((T*)a.h_out + row * a.h_row + (int64_t)v * V, pack<T, V>(f));
#pragma unroll
        for (int j = 0; j < V; ++j) sum = fmaf(f[j], f[j], sum);
        if constexpr (kFp8) {
          float g[V];
          unpack<T, V>(kAhead ? w[i] : weight(i), g);
#pragma unroll
          for (int j = 0; j < V; ++j) top = fmaxf(top, fabsf(f[j] * g[j]));
        }
      }
    }
    const float2 all = row_reduce<true>(sum, top, s_red, turn);
    const float r = rsqrtf(fmaf(all.x, inv_width, a.eps));
    Fp8Row q8{};
    if constexpr (kFp8) {
      q8 = fp8_row(all.y, r);
      if (live && threadIdx.x == 0) a.scale[row] = q8.scale;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (live && v < vecs) {
        float f[V], g[V];
        sum_of(i, f);
        unpack<T, V>(kAhead ? w[i] : weight(i), g);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = kFp8 ? q8(f[j], g[j]) : f[j] * (r * g[j]);
        if constexpr (!kFp8) {
          store_pack<T, V>((T*)a.y + row * a.y_row + (int64_t)v * V, pack<T, V>(f));
        } else {
          uint8_t* dst = (uint8_t*)a.y + row * a.y_row + (int64_t)v * V;
          if constexpr (V == 1) {
            *dst = __nv_cvt_float_to_fp8(f[0], __NV_SATFINITE, __NV_E4M3);
          } else {
            uint32_t word[V / 4];
#pragma unroll
            for (int j = 0; j < V; j += 4) {
              const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[j], f[j + 1]), __NV_SATFINITE, __NV_E4M3);
              const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[j + 2], f[j + 3]), __NV_SATFINITE, __NV_E4M3);
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

// r^3 mean(w dy h), the factor of h in dx: r^3 alone is beyond 32 bits for rows
// of small values under a small eps (r above 7e12), the mean being as small.
__device__ __forceinline__ float norm_along(float r, float mean) { return r * mean * r * r; }

// Rows of dx, and a block's part of dweight in registers over its rows: part
// [blocks, width] in the workspace, summed by k_norm_weight in a fixed order.
template <class T, int V, int NV>
__global__ void __launch_bounds__(kMaxThreads) k_norm_backward(NormBackwardLaunch n) {
  let_next_kernel_start();
  const tb_norm_backward_args& a = n.a;
  extern __shared__ float s_part[];  // [rows, per_row * NV * V] where a block has more than one row
  __shared__ float2 s_red[64];
  int turn = 0;
  const int vecs = a.width / V;
  const float inv_width = 1.f / (float)a.width;
  const int64_t stride = (int64_t)gridDim.x * blockDim.y;
  constexpr bool kAhead = ahead<T, V, NV, true>();
  float dw[NV][V] = {};
  Pack<T, V> w[NV], ph[NV], pd[NV], pg[NV];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (row < a.rows && v < vecs) {
        ph[i] = load_pack<T, V>((const T*)a.h + row * a.h_row + (int64_t)v * V);
        pd[i] = load_pack<T, V>((const T*)a.dy + row * a.dy_row + (int64_t)v * V);
        if (a.dh) pg[i] = load_pack<T, V>((const T*)a.dh + row * a.dh_row + (int64_t)v * V);
      }
    }
  };
  int64_t base = (int64_t)blockIdx.x * blockDim.y;
  if (kAhead) load(base + threadIdx.y);
  auto weight = [&](int i) { return load_pack<T, V>((const T*)a.weight + (int64_t)(threadIdx.x + i * blockDim.x) * V); };
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (kAhead && threadIdx.x + i * blockDim.x < vecs) w[i] = weight(i);
  for (; base < a.rows; base += stride) {
    const int64_t row = base + threadIdx.y;
    const bool live = row < a.rows;
    Pack<T, V> ch[NV], cd[NV], cg[NV];
    if (!kAhead) load(row);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      ch[i] = ph[i];
      cd[i] = pd[i];
      cg[i] = pg[i];
    }
    if (kAhead) load(row + stride);
    float hh = 0.f, hd = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (live && v < vecs) {
        float h[V], d[V], g[V];
        unpack<T, V>(ch[i], h);
        unpack<T, V>(cd[i], d);
        unpack<T, V>(kAhead ? w[i] : weight(i), g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          hh = fmaf(h[j], h[j], hh);
          hd = fmaf(h[j] * g[j], d[j], hd);
        }
      }
    }
    const float2 all = row_reduce<false>(hh, hd, s_red, turn);
    const float r = rsqrtf(fmaf(all.x, inv_width, a.eps));
    const float m = norm_along(r, all.y * inv_width);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (live && v < vecs) {
        float h[V], d[V], f[V], g[V];
        unpack<T, V>(ch[i], h);
        unpack<T, V>(cd[i], d);
        unpack<T, V>(kAhead ? w[i] : weight(i), f);
        if (a.dh) unpack<T, V>(cg[i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          dw[i][j] = fmaf(d[j], h[j] * r, dw[i][j]);
          const float x = fmaf(-m, h[j], r * f[j] * d[j]);
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

// ------------------------------------------- rows that no vector boundary meets
//
// A row of an odd width starts anywhere in a vector of 16 bytes.  Blocks move
// groups of whole rows of a dense tensor through shared memory by the vectors
// they lie in, the next group while one is normed, and read single elements
// there (50000 rows of 777 in 16 bits: 49 us, 82 element by element; the
// gradient 81 us and 141).  A group has up to 16 / sizeof(T) rows, a whole
// number of vectors; fewer, with more warps each, where rows are wide.
constexpr int kGroupWarps = 32;  // at most

__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// Rows [row, row + rows) of a dense tensor of `all` rows, on their way into
// `dst`, as far into a vector as they lie in theirs: that offset, in elements.
// The vectors at the ends come whole, but for the tensor's last.
template <class T>
__device__ __forceinline__ int group_phase(int64_t row, int width) {
  return (int)(row * width % (16 / (int)sizeof(T)));
}
template <class T>
__device__ __forceinline__ void fetch_group(T* dst, const void* src, int64_t row, int rows, int64_t all, int width) {
  constexpr int G = 16 / (int)sizeof(T);
  const int phase = group_phase<T>(row, width);
  const T* from = (const T*)src + row * width - phase;
  const int end = phase + (int)min((int64_t)rows, all - row) * width;
  const int64_t last = phase + (all - row) * width;
  for (int i = threadIdx.x * G; i < end; i += blockDim.x * G) {
    if (i + G <= last) copy_async(dst + i, from + i);
    else
      for (int j = i; j < end; ++j) dst[j] = from[j];
  }
}
template <class T>
__device__ __forceinline__ void put_group(void* dst, const T* src, int64_t row, int rows, int64_t all, int width) {
  constexpr int G = 16 / (int)sizeof(T);
  const int phase = group_phase<T>(row, width);
  T* to = (T*)dst + row * width - phase;
  const int end = phase + (int)min((int64_t)rows, all - row) * width;
  for (int i = threadIdx.x * G; i < end; i += blockDim.x * G) {
    if (i >= phase && i + G <= end) *reinterpret_cast<uint4*>(to + i) = *reinterpret_cast<const uint4*>(src + i);
    else
      for (int j = max(i, phase); j < min(i + G, end); ++j) to[j] = src[j];
  }
}

// Sums (the second one: sum or maximum) over the warps of each row of a group.
template <bool kMax>
__device__ __forceinline__ float2 group_reduce(float x, float y, float2* s, int per_row) {
  x = warp_sum(x);
  y = kMax ? warp_max(y) : warp_sum(y);
  if (per_row == 1) return make_float2(x, y);
  const int warp = threadIdx.x >> 5, first = warp / per_row * per_row;
  if ((threadIdx.x & 31) == 0) s[warp] = make_float2(x, y);
  __syncthreads();
  float2 v = s[first];
  for (int i = 1; i < per_row; ++i) {
    v.x += s[first + i].x;
    v.y = kMax ? fmaxf(v.y, s[first + i].y) : v.y + s[first + i].y;
  }
  return v;
}

// Shared memory: the weight, then `nv` buffers of a group of x, residual.
template <class T, bool kFp8>
__global__ void __launch_bounds__(32 * kGroupWarps) k_norm_groups(NormLaunch n) {
  const tb_norm_args& a = n.a;
  extern __shared__ __align__(16) char s_group[];
  __shared__ float2 s_red[kGroupWarps];
  const int width = a.width, per_row = (int)(blockDim.x >> 5) / n.rows, g = (threadIdx.x >> 5) / per_row;
  const int first = threadIdx.x - g * per_row * 32, step = per_row * 32;
  const int tensors = a.residual ? 2 : 1;
  const int span = (int)(norm_buffer_bytes(width, sizeof(T), n.rows) / sizeof(T));
  T* w = reinterpret_cast<T*>(s_group);
  T* buf = w + up_to(width, 16 / (int)sizeof(T));
  const float inv_width = 1.f / (float)width;
  const int64_t stride = (int64_t)gridDim.x * n.rows;
  for (int i = threadIdx.x; i < width; i += blockDim.x) w[i] = ((const T*)a.weight)[i];
  auto fetch = [&](int64_t base, int st) {
    if (base < a.rows) {
      T* to = buf + (size_t)st * tensors * span;
      fetch_group(to, a.x, base, n.rows, a.rows, width);
      if (a.residual) fetch_group(to + span, a.residual, base, n.rows, a.rows, width);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int st = 0;
  if (n.nv > 1) fetch((int64_t)blockIdx.x * n.rows, 0);
  for (int64_t base = (int64_t)blockIdx.x * n.rows; base < a.rows; base += stride) {
    if (n.nv > 1) {
      fetch(base + stride, st ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      fetch(base, 0);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    T* x = buf + (size_t)st * tensors * span;
    T* res = x + span;
    const int64_t row = base + g;
    const int at = group_phase<T>(base, width) + g * width;
    const int mine = row < a.rows ? width : 0;
    float sum = 0.f, top = 0.f;
    for (int i = first; i < mine; i += step) {
      float f = RowType<T>::to(x[at + i]);
      if (a.residual) f += RowType<T>::to(res[at + i]);
      sum = fmaf(f, f, sum);
      if (kFp8) top = fmaxf(top, fabsf(f * RowType<T>::to(w[i])));
    }
    const float2 all = group_reduce<true>(sum, top, s_red, per_row);
    const float r = rsqrtf(fmaf(all.x, inv_width, a.eps));
    const Fp8Row q8 = kFp8 ? fp8_row(all.y, r) : Fp8Row{};
    if (kFp8 && first == 0 && mine) a.scale[row] = q8.scale;
    uint8_t* q = (uint8_t*)a.y + row * width;
    for (int i = first; i < mine; i += step) {
      float f = RowType<T>::to(x[at + i]);
      if (a.residual) {
        f += RowType<T>::to(res[at + i]);
        res[at + i] = RowType<T>::from(f);
      }
      const float g = RowType<T>::to(w[i]);
      if (kFp8) q[i] = __nv_cvt_float_to_fp8(q8(f, g), __NV_SATFINITE, __NV_E4M3);
      else x[at + i] = RowType<T>::from(f * (r * g));
    }
    __syncthreads();
    if (!kFp8) put_group(a.y, x, base, n.rows, a.rows, width);
    if (a.h_out) put_group(a.h_out, res, base, n.rows, a.rows, width);
    if (n.nv > 1) st ^= 1;
    __syncthreads();  // the group's buffer may be filled again
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Shared memory: the weight and dweight's part in 32 bits, then `nv` buffers
// of a group of h, dy, dh; dx takes dy's place.
template <class T>
__global__ void __launch_bounds__(32 * kGroupWarps) k_norm_backward_groups(NormBackwardLaunch n) {
  let_next_kernel_start();
  const tb_norm_backward_args& a = n.a;
  extern __shared__ __align__(16) char s_group[];
  __shared__ float2 s_red[kGroupWarps], s_row[8];  // r and the factor of h
  const int width = a.width, per_row = (int)(blockDim.x >> 5) / n.rows, g = (threadIdx.x >> 5) / per_row;
  const int first = threadIdx.x - g * per_row * 32, step = per_row * 32;
  const int tensors = a.dh ? 3 : 2;
  const int span = (int)(norm_buffer_bytes(width, sizeof(T), n.rows) / sizeof(T));
  float* w = reinterpret_cast<float*>(s_group);
  float* dw = w + up_to(width, 4);
  T* buf = reinterpret_cast<T*>(dw + up_to(width, 4));
  const float inv_width = 1.f / (float)width;
  const int64_t stride = (int64_t)gridDim.x * n.rows;
  for (int i = threadIdx.x; i < width; i += blockDim.x) {
    w[i] = RowType<T>::to(((const T*)a.weight)[i]);
    dw[i] = 0.f;
  }
  auto fetch = [&](int64_t base, int st) {
    if (base < a.rows) {
      T* to = buf + (size_t)st * tensors * span;
      fetch_group(to, a.h, base, n.rows, a.rows, width);
      fetch_group(to + span, a.dy, base, n.rows, a.rows, width);
      if (a.dh) fetch_group(to + 2 * span, a.dh, base, n.rows, a.rows, width);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int st = 0;
  if (n.nv > 1) fetch((int64_t)blockIdx.x * n.rows, 0);
  for (int64_t base = (int64_t)blockIdx.x * n.rows; base < a.rows; base += stride) {
    if (n.nv > 1) {
      fetch(base + stride, st ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      fetch(base, 0);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const int phase = group_phase<T>(base, width);
    T* h = buf + (size_t)st * tensors * span + phase;
    T* d = h + span;
    const T* dh = d + span;
    const int rows = (int)min((int64_t)n.rows, a.rows - base);
    const int mine = g < rows ? width : 0;
    float hh = 0.f, hd = 0.f;
    for (int i = first; i < mine; i += step) {
      const float f = RowType<T>::to(h[g * width + i]);
      hh = fmaf(f, f, hh);
      hd = fmaf(f * w[i], RowType<T>::to(d[g * width + i]), hd);
    }
    const float2 all = group_reduce<false>(hh, hd, s_red, per_row);
    const float r = rsqrtf(fmaf(all.x, inv_width, a.eps));
    if (first == 0) s_row[g] = make_float2(r, -norm_along(r, all.y * inv_width));
    __syncthreads();
    // by columns: a thread's part of dweight stays its own
    for (int i = threadIdx.x; i < width; i += blockDim.x) {
      const float wi = w[i];
      float sum = dw[i];
#pragma unroll 4
      for (int k = 0; k < rows; ++k) {
        const float2 rm = s_row[k];
        const float f = RowType<T>::to(h[k * width + i]), e = RowType<T>::to(d[k * width + i]);
        sum = fmaf(e, f * rm.x, sum);
        float x = fmaf(rm.y, f, rm.x * wi * e);
        if (a.dh) x += RowType<T>::to(dh[k * width + i]);
        d[k * width + i] = RowType<T>::from(x);
      }
      dw[i] = sum;
    }
    __syncthreads();
    put_group(a.dx, d - phase, base, n.rows, a.rows, width);
    if (n.nv > 1) st ^= 1;
    __syncthreads();  // the group's buffer may be filled again
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  for (int i = threadIdx.x; i < width; i += blockDim.x) a.workspace[(int64_t)blockIdx.x * width + i] = dw[i];
}

// dweight = the blocks' parts summed, in a fixed order: 8 columns a block, 64
// rows of parts at a time, four in flight a thread.
template <class T>
__global__ void __launch_bounds__(512) k_norm_weight(NormBackwardLaunch n) {
  constexpr int kCols = 8, kRows = 64;
  __shared__ float s[kRows][kCols + 1];
  const int x = threadIdx.x % kCols, y = threadIdx.x / kCols, c = blockIdx.x * kCols + x;
  wait_for_last_kernel();
  float sum = 0.f;
  if (c < n.a.width) {
    const float* part = n.a.workspace + c;
    int b = y;
    for (; b + 3 * kRows < n.blocks; b += 4 * kRows) {
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = part[(int64_t)(b + i * kRows) * n.a.width];
      sum += (f[0] + f[1]) + (f[2] + f[3]);
    }
    for (; b < n.blocks; b += kRows) sum += part[(int64_t)b * n.a.width];
  }
  s[y][x] = sum;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < kCols) {
    const float all = warp_sum(s[lane][warp] + s[lane + 32][warp]);
    const int o = blockIdx.x * kCols + warp;
    if (lane == 0 && o < n.a.width) ((T*)n.a.dweight)[o] = RowType<T>::from(all);
  }
}

template <class T, bool kFp8>
cudaError_t go_groups(const NormLaunch& n, cudaStream_t s) {
  const size_t bytes = norm_group_bytes(n.a.width, sizeof(T), n.a.residual ? 2 : 1, n.rows, n.nv, sizeof(T));
  static std::atomic<bool> ready[kMaxDevices];
  const cudaError_t e = allow_shared(k_norm_groups<T, kFp8>, kNormGroupBytes, ready);
  if (e != cudaSuccess) return e;
  k_norm_groups<T, kFp8><<<n.blocks, n.per_row, bytes, s>>>(n);
  return cudaGetLastError();
}
template <class T>
cudaError_t go_back_groups(const NormBackwardLaunch& n, cudaStream_t s) {
  const size_t bytes = norm_group_bytes(n.a.width, sizeof(T), n.a.dh ? 3 : 2, n.rows, n.nv, 8);
  static std::atomic<bool> ready[kMaxDevices];
  const cudaError_t e = allow_shared(k_norm_backward_groups<T>, kNormGroupBytes, ready);
  if (e != cudaSuccess) return e;
  k_norm_backward_groups<T><<<n.blocks, n.per_row, bytes, s>>>(n);
  return cudaGetLastError();
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
  if (n.groups) return n.a.fp8 ? go_groups<T, true>(n, s) : go_groups<T, false>(n, s);
  if (n.vec) {
    switch (n.nv) {
      case 1: return go<T, V, 1>(n, s);
      case 2: return go<T, V, 2>(n, s);
      case 4: return go<T, V, 4>(n, s);
      default: return go<T, V, 8>(n, s);
    }
  }
  switch (n.nv) {
    case 4: return go<T, 1, 4>(n, s);
    case 8: return go<T, 1, 8>(n, s);
    default: return go<T, 1, 32>(n, s);
  }
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
  if (n.groups) return go_back_groups<T>(n, s);
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
  auto go = [&](auto kernel) { return launch_early(kernel, (n.a.width + 7) / 8, 512, 0, s, n.a.rows > 0, n); };
  switch (n.a.type) {
    case TB_TYPE_F32: return go(k_norm_weight<float>);
    case TB_TYPE_F16: return go(k_norm_weight<__half>);
    default: return go(k_norm_weight<__nv_bfloat16>);
  }
}

}  // namespace tb
