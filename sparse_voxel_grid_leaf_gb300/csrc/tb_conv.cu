// Short causal convolution of every channel over jagged rows, its gradient and
// its step for single rows (tb_causal_conv, tb_causal_conv_backward,
// tb_causal_conv_step).
//
//   pre_t = bias + sum_j weight[c, j] x_(t - taps + 1 + j),  y = pre sigmoid(pre)
//
// Every element is read once and written once, so the bound is memory.  A
// thread walks down a run of rows with a vector of channels and keeps the last
// taps - 1 rows in registers; what a run reads of the run before is taps - 1
// rows.  The gradient walks with two windows, of x and of the gradient of pre:
// dx_t is known once the gradient of pre at t + taps - 1 is.
//
// Measured, bf16, 4 taps and SiLU: 124807 rows of 1024 channels 87 us, 5.9 TB/s
// (127 with four rows ahead in registers and runs of 32 rows, whose first loads
// one after another took a quarter; 99 with fours of rows and a rest, where
// eight with an early end are one loop); the gradient of 60013 rows of 1536 115 us,
// 4.8 TB/s (162 while every row asked whether it was the run's own).
#include "tb_seq.cuh"
#include "tb_seq.h"

#include <type_traits>

namespace tb {
namespace {

constexpr int kConvThreads = 128;  // of a block at most

__device__ __forceinline__ void conv_grid(const tb_conv_args& a, int b, int64_t& begin, int64_t& end) {
  if (!a.offsets) {
    begin = 0;
    end = a.tokens;
    return;
  }
  begin = min(max(a.offsets[b], (int64_t)0), a.tokens);
  end = min(max(a.offsets[b + 1], begin), a.tokens);
}

// The last grid that starts at or before a row; -1: none.
__device__ __forceinline__ int conv_grid_of(const tb_conv_args& a, int64_t row) {
  if (!a.offsets) return 0;
  int lo = -1, hi = a.grids;  // offsets[lo] <= row < offsets[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.offsets[mid] <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The pieces of the rows [at, end) that lie in one grid, or in none (grid -1).
struct ConvPieces {
  const tb_conv_args& a;
  int64_t at, end;
  int b;
  int64_t begin = 0, past = 0;  // the piece's grid
  __device__ ConvPieces(const tb_conv_args& a, int64_t at, int64_t end) : a(a), at(at), end(end), b(conv_grid_of(a, at)) {}
  // [r0, r1) of the next piece; the grid or -1
  __device__ __forceinline__ int next(int64_t& r0, int64_t& r1) {
    r0 = at;
    while (true) {
      if (b >= 0) {
        conv_grid(a, b, begin, past);
        if (at >= begin && at < past) {
          r1 = at = min(past, end);
          return b;
        }
      }
      if (b + 1 >= a.grids) break;
      if (b + 1 >= 0) {
        int64_t from, to;
        conv_grid(a, b + 1, from, to);
        if (from > at) {
          r1 = at = min(from, end);
          return -1;
        }
      }
      ++b;
    }
    r1 = at = end;
    return -1;
  }
};

// Row `place` of grid b, of its state where place < 0.
template <class T, int V, int K>
__device__ __forceinline__ Pack<T, V> conv_row(const tb_conv_args& a, int b, int64_t begin, int64_t place, int c) {
  Pack<T, V> r{};
  if (place >= 0) return load_pack<T, V>((const T*)a.x + (begin + place) * a.x_row + c);
  if (a.state) r = load_pack<T, V>((const T*)a.state + ((int64_t)b * (K - 1) + (K - 1) + place) * a.channels + c);
  return r;
}

template <class T, int V, int K>
struct ConvWeight {
  static constexpr int P = (V + 1) / 2;
  f32x2 w[K][P], bias[P];
  __device__ __forceinline__ ConvWeight(const void* weight, const void* b, int c) {
    float f[V * K], g[V] = {};  // a vector's channels and taps are consecutive, and whole vectors
    constexpr int U = V > 1 ? 8 / (int)sizeof(T) : 1;
#pragma unroll
    for (int i = 0; i < V * K; i += U) {
      float u[U];
      unpack<T, U>(load_pack<T, U>((const T*)weight + (int64_t)c * K + i), u);
#pragma unroll
      for (int k = 0; k < U; ++k) f[i + k] = u[k];
    }
    if (b) unpack<T, V>(load_pack<T, V>((const T*)b + c), g);
    auto at = [&](int v, int k) { return f[v * K + k]; };
    auto of = [&](int v) { return g[v]; };
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const int second = V > 1 ? v + 1 : v;
#pragma unroll
      for (int k = 0; k < K; ++k) w[k][v / 2] = pair(at(v, k), at(second, k));
      bias[v / 2] = pair(of(v), of(second));
    }
  }
};

// sigmoid(x) = 1 / (1 + exp(-x)): at the ends of the range the exponential is 0
// or infinite and the quotient 1 or 0.
__device__ __forceinline__ f32x2 sigmoid(f32x2 x) {
  const float2 e = halves(mul2(x, both(-1.4426950408889634f)));
  float2 u;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(u.x) : "f"(e.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(u.y) : "f"(e.y));
  const float2 w = halves(add2(pair(u.x, u.y), both(1.f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(u.x) : "f"(w.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(u.y) : "f"(w.y));
  return pair(u.x, u.y);
}

// N tensors' rows on their way to a thread, `kAhead` rows ahead: each thread's
// own, through shared memory by asynchronous copies (registers for as many
// would leave too few threads), or four rows in registers where a vector is
// smaller than such a copy.
template <class T, int V, int N>
struct RowsAhead {
  static constexpr bool kShared = V * sizeof(T) >= 4;
  static constexpr int kSlots = kShared ? 16 : 4;
  static constexpr int kBytes = kShared ? kSlots * N * kConvThreads * V * (int)sizeof(T) : 16;
  Pack<T, V> held[kShared ? 1 : kSlots][N];
  Pack<T, V>* mine;
  const T* next[N];  // row `asked`
  int64_t stride[N];
  int asked, have;   // rows on their way or taken, of all
  __device__ __forceinline__ void ask() {
    if (asked < have) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(mine + (asked % kSlots * N + n) * kConvThreads);
        if constexpr (V * sizeof(T) == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(next[n]) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(next[n]), "n"(V * sizeof(T)) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void more(int i) {
    if constexpr (kShared) {
      ask();
    } else if (asked < have) {
#pragma unroll
      for (int n = 0; n < N; ++n) held[i][n] = load_pack<T, V>(next[n]);
    }
    ++asked;
#pragma unroll
    for (int n = 0; n < N; ++n) next[n] += stride[n];
  }
  __device__ __forceinline__ void start(int rows) {
    have = rows;
    asked = 0;
#pragma unroll
    for (int u = 0; u < (kShared ? kSlots - 1 : kSlots); ++u) more(u);
  }
  // Row u < have; i = u % 4, known to the compiler.
  __device__ __forceinline__ void take(int u, int i, Pack<T, V> (&row)[N]) {
    if constexpr (kShared) asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 2) : "memory");
#pragma unroll
    for (int n = 0; n < N; ++n) row[n] = kShared ? mine[(u % kSlots * N + n) * kConvThreads] : held[kShared ? 0 : i][n];
    more(i);
  }
  // The rows have been taken, and the slots may be filled again.
  __device__ __forceinline__ void finish() {
    if constexpr (kShared) asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
};

// The last taps - 1 rows of state and grid together.
template <class T, int V, int K>
__device__ __forceinline__ void conv_last(const tb_conv_args& a, int b, int c) {
  int64_t begin, end;
  conv_grid(a, b, begin, end);
#pragma unroll
  for (int i = 0; i < K - 1; ++i)
    store_pack<T, V>((T*)a.state_out + ((int64_t)b * (K - 1) + i) * a.channels + c,
                     conv_row<T, V, K>(a, b, begin, end - begin - (K - 1) + i, c));
}

// Blocks along the rows and the channels: blockIdx.x = rows' block * blocks_x + channels' block.
template <class T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) k_conv(ConvLaunch l) {
  const tb_conv_args& a = l.a;
  const int bx = (int)(blockIdx.x % l.blocks_x), per_y = (int)blockDim.x / l.per_x;
  const int64_t by = blockIdx.x / l.blocks_x;
  const int c = (bx * l.per_x + (int)threadIdx.x % l.per_x) * V, y = (int)threadIdx.x / l.per_x;
  if (c >= a.channels || y >= per_y) return;
  const int64_t run = by * per_y + y;
  if (run >= l.runs) {
    if (a.state_out && run - l.runs < a.grids) conv_last<T, V, K>(a, (int)(run - l.runs), c);
    return;
  }
  __shared__ __align__(16) char s_ahead[RowsAhead<T, V, 1>::kBytes];
  RowsAhead<T, V, 1> ahead;
  ahead.mine = reinterpret_cast<Pack<T, V>*>(s_ahead) + threadIdx.x;
  ahead.stride[0] = a.x_row;
  const ConvWeight<T, V, K> w(a.weight, a.bias, c);
  constexpr int P = (V + 1) / 2;  // pairs of channels
  ConvPieces pieces(a, run * l.run, min((run + 1) * l.run, a.tokens));
  while (pieces.at < pieces.end) {
    int64_t r0, r1;
    const int b = pieces.next(r0, r1);
    T* to = (T*)a.y + r0 * a.y_row + c;
    if (b < 0) {
      for (int64_t r = r0; r < r1; ++r, to += a.y_row) store_pack<T, V>(to, Pack<T, V>{});
      continue;
    }
    const int n = (int)(r1 - r0);
    ahead.next[0] = (const T*)a.x + r0 * a.x_row + c;
    ahead.start(n);
    f32x2 x[K][P];  // the rows before, oldest first, and the row
#pragma unroll
    for (int i = 0; i < K - 1; ++i) to_pairs<T, V>(conv_row<T, V, K>(a, b, pieces.begin, r0 - pieces.begin - (K - 1) + i, c), x[i]);
    auto step = [&](int u, int i) {
      Pack<T, V> row[1];
      f32x2 o[P];
      ahead.take(u, i, row);
      to_pairs<T, V>(row[0], x[K - 1]);
#pragma unroll
      for (int v = 0; v < P; ++v) {
        f32x2 s = w.bias[v];
#pragma unroll
        for (int k = 0; k < K; ++k) s = fma2(w.w[k][v], x[k][v], s);
        o[v] = a.silu ? mul2(s, sigmoid(s)) : s;
#pragma unroll
        for (int k = 0; k < K - 1; ++k) x[k][v] = x[k + 1][v];
      }
      store_pack<T, V>(to, from_pairs<T, V>(o));
      to += a.y_row;
    };
    for (int base = 0; base < n; base += 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (base + i >= n) break;
        step(base + i, i % 4);
      }
    }
    ahead.finish();
  }
}

// The gradient of pre from that of y.
__device__ __forceinline__ f32x2 conv_slope(f32x2 dy, f32x2 pre, int silu) {
  if (!silu) return dy;
  const f32x2 s = sigmoid(pre), rest = fma2(s, both(-1.f), both(1.f));
  return mul2(dy, mul2(s, fma2(pre, rest, both(1.f))));
}

// The gradient of a grid's first state: its row m is the tap m - p of the row at
// place p, and in a grid of fewer than taps - 1 rows part of the last state.
template <class T, int V, int K>
__device__ __forceinline__ void conv_first(const ConvBackwardLaunch& l, int b, int c) {
  constexpr int P = (V + 1) / 2;
  const tb_conv_args& a = l.f.a;
  const tb_conv_backward_args& g = l.g;
  int64_t begin, end;
  conv_grid(a, b, begin, end);
  const ConvWeight<T, V, K> w(a.weight, a.bias, c);
  f32x2 sum[K - 1][P] = {}, x[2 * K - 2][P];
#pragma unroll
  for (int i = 0; i < 2 * K - 2; ++i) {
    Pack<T, V> p{};
    if (i - (K - 1) < end - begin) p = conv_row<T, V, K>(a, b, begin, i - (K - 1), c);
    to_pairs<T, V>(p, x[i]);
  }
#pragma unroll
  for (int p = 0; p < K - 1; ++p) {
    if (p >= end - begin) break;
    f32x2 dy[P];
    to_pairs<T, V>(load_pack<T, V>((const T*)g.dy + (begin + p) * g.dy_row + c), dy);
#pragma unroll
    for (int v = 0; v < P; ++v) {
      f32x2 s = w.bias[v];
#pragma unroll
      for (int k = 0; k < K; ++k) s = fma2(w.w[k][v], x[p + k][v], s);
      const f32x2 d = conv_slope(dy[v], s, a.silu);
#pragma unroll
      for (int m = p; m < K - 1; ++m) sum[m][v] = fma2(w.w[m - p][v], d, sum[m][v]);
    }
  }
#pragma unroll
  for (int m = 0; m < K - 1; ++m) {
    const int64_t i = m - (end - begin);
    if (g.dstate_out && i >= 0) {
      f32x2 f[P];
      to_pairs<T, V>(load_pack<T, V>((const T*)g.dstate_out + ((int64_t)b * (K - 1) + i) * a.channels + c), f);
#pragma unroll
      for (int v = 0; v < P; ++v) sum[m][v] = add2(sum[m][v], f[v]);
    }
    store_pack<T, V>((T*)g.dstate + ((int64_t)b * (K - 1) + m) * a.channels + c, from_pairs<T, V>(sum[m]));
  }
}

// Parts of dweight and dbias in registers over a run, joined over a block's
// runs in shared memory: part [parts, taps + 1, channels] in the workspace.
template <class T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) k_conv_backward(ConvBackwardLaunch l) {
  let_next_kernel_start();
  const tb_conv_args& a = l.f.a;
  const tb_conv_backward_args& g = l.g;
  __shared__ f32x2 s_part[kConvThreads][(V + 1) / 2];
  const int bx = (int)(blockIdx.x % l.f.blocks_x), per_x = l.f.per_x, per_y = (int)blockDim.x / per_x;
  const int64_t by = blockIdx.x / l.f.blocks_x;
  const int c = (bx * per_x + (int)threadIdx.x % per_x) * V, y = (int)threadIdx.x / per_x;
  const bool live = c < a.channels && y < per_y;
  if (by >= l.parts) {  // a block of grids
    const int64_t b = (by - l.parts) * per_y + y;
    if (live && b < a.grids) conv_first<T, V, K>(l, (int)b, c);
    return;
  }
  const int64_t run = by * per_y + y;
  constexpr int P = (V + 1) / 2;
  f32x2 dw[K + 1][P] = {};  // the last one: dbias
  __shared__ __align__(16) char s_ahead[RowsAhead<T, V, 2>::kBytes];
  if (live && run < l.f.runs) {
    const ConvWeight<T, V, K> w(a.weight, a.bias, c);
    RowsAhead<T, V, 2> ahead;
    ahead.mine = reinterpret_cast<Pack<T, V>*>(s_ahead) + threadIdx.x;
    ahead.stride[0] = a.x_row, ahead.stride[1] = g.dy_row;
    ConvPieces pieces(a, run * l.f.run, min((run + 1) * l.f.run, a.tokens));
    while (pieces.at < pieces.end) {
      int64_t r0, r1;
      const int b = pieces.next(r0, r1);
      T* to = (T*)g.dx + r0 * g.dx_row + c;
      if (b < 0) {
        for (int64_t r = r0; r < r1; ++r, to += g.dx_row) store_pack<T, V>(to, Pack<T, V>{});
        continue;
      }
      f32x2 x[K][P], d[K][P] = {};  // rows of x and gradients of pre, the last one at [K - 1]
#pragma unroll
      for (int i = 0; i < K - 1; ++i) to_pairs<T, V>(conv_row<T, V, K>(a, b, pieces.begin, r0 - pieces.begin - (K - 1) + i, c), x[i]);
      const int own = (int)(r1 - r0);                                     // rows of the run
      const int have = (int)min(pieces.past - r0, (int64_t)own + K - 1);  // rows whose pre has a part in them
      ahead.next[0] = (const T*)a.x + r0 * a.x_row + c;
      ahead.next[1] = (const T*)g.dy + r0 * g.dy_row + c;
      ahead.start(have);
      // Row u of x and dy in, row u - (K - 1) of dx out.  kWhole: both are the
      // run's own, and dx's has K - 1 rows of its grid behind it.
      auto step = [&](int u, int i, auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
        if (kWhole || u < have) {
          Pack<T, V> row[2];
          f32x2 e[P];
          ahead.take(u, i, row);
          to_pairs<T, V>(row[0], x[K - 1]);
          to_pairs<T, V>(row[1], e);
#pragma unroll
          for (int v = 0; v < P; ++v) {
            f32x2 s = w.bias[v];
#pragma unroll
            for (int k = 0; k < K; ++k) s = fma2(w.w[k][v], x[k][v], s);
            d[K - 1][v] = conv_slope(e[v], s, a.silu);
          }
          if (kWhole || u < own) {
#pragma unroll
            for (int v = 0; v < P; ++v) {
#pragma unroll
              for (int k = 0; k < K; ++k) dw[k][v] = fma2(d[K - 1][v], x[k][v], dw[k][v]);
              dw[K][v] = add2(dw[K][v], d[K - 1][v]);
            }
          }
        } else {
#pragma unroll
          for (int v = 0; v < P; ++v) d[K - 1][v] = 0;
        }
        if (kWhole || u >= K - 1) {
          f32x2 o[P];
#pragma unroll
          for (int v = 0; v < P; ++v) {
            o[v] = mul2(w.w[K - 1][v], d[0][v]);
#pragma unroll
            for (int k = 1; k < K; ++k) o[v] = fma2(w.w[K - 1 - k][v], d[k][v], o[v]);
          }
          if (!kWhole) {
            const int64_t left = pieces.past - 1 - (r0 + u - (K - 1));
            if (g.dstate_out && left < K - 1) {
              f32x2 f[P];
              to_pairs<T, V>(load_pack<T, V>((const T*)g.dstate_out + ((int64_t)b * (K - 1) + K - 2 - left) * a.channels + c), f);
#pragma unroll
              for (int v = 0; v < P; ++v) o[v] = add2(o[v], f[v]);
            }
          }
          store_pack<T, V>(to, from_pairs<T, V>(o));
          to += g.dx_row;
        }
#pragma unroll
        for (int v = 0; v < P; ++v)
#pragma unroll
          for (int k = 0; k < K - 1; ++k) {
            x[k][v] = x[k + 1][v];
            d[k][v] = d[k + 1][v];
          }
      };
      const int all = own + K - 1;
      int u = 0;
      while (u < all) {  // four rows at a time
        if (u >= K - 1 && u + 4 <= own) {
#pragma unroll
          for (int i = 0; i < 4; ++i) step(u + i, i, std::true_type());
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (u + i < all) step(u + i, i, std::false_type());
        }
        u += 4;
      }
      ahead.finish();
    }
  }
  float* part = g.workspace + by * (K + 1) * a.channels + c;
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    if (per_y > 1) {
      if (k) __syncthreads();
#pragma unroll
      for (int v = 0; v < P; ++v) s_part[threadIdx.x][v] = dw[k][v];
      __syncthreads();
      if (y == 0)
        for (int i = 1; i < per_y; ++i)
#pragma unroll
          for (int v = 0; v < P; ++v) dw[k][v] = add2(dw[k][v], s_part[threadIdx.x + i * per_x][v]);
    }
    if (live && y == 0)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 f = halves(dw[k][v / 2]);
        part[(int64_t)k * a.channels + v] = v % 2 ? f.y : f.x;
      }
  }
}

// dweight and dbias = the blocks' parts summed, in a fixed order: 32 columns a block.
template <class T>
__global__ void __launch_bounds__(512) k_conv_weight(ConvBackwardLaunch l) {
  __shared__ float s[16][33];
  const int K = l.f.a.taps, C = l.f.a.channels;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t width = (int64_t)(K + 1) * C, o = (int64_t)blockIdx.x * 32 + x;
  wait_for_last_kernel();
  float sum = 0.f;
  if (o < width) {
    const float* part = l.g.workspace + o;
    int64_t p = y;
    for (; p + 48 < l.parts; p += 64) {
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = part[(p + 16 * i) * width];
      sum += (f[0] + f[1]) + (f[2] + f[3]);
    }
    for (; p < l.parts; p += 16) sum += part[p * width];
  }
  s[y][x] = sum;
  __syncthreads();
  if (y == 0 && o < width) {
#pragma unroll
    for (int i = 1; i < 16; ++i) sum += s[i][x];
    const int64_t k = o / C, c = o - k * C;
    if (k < K) ((T*)l.g.dweight)[c * K + k] = RowType<T>::from(sum);
    else if (l.g.dbias) ((T*)l.g.dbias)[c] = RowType<T>::from(sum);
  }
}

template <class T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) k_conv_step(ConvStepLaunch l) {
  const tb_conv_step_args& a = l.a;
  const int cols = a.channels / V;
  const int64_t at = (int64_t)blockIdx.x * kConvThreads + threadIdx.x, n = at / cols;
  if (n >= a.streams) return;
  const int c = (int)(at - n * cols) * V;
  const int64_t slot = a.slots ? (int64_t)a.slots[n] : n;
  T* to = (T*)a.y + n * a.y_row + c;
  if (slot < 0 || slot >= a.num_slots) {
    store_pack<T, V>(to, Pack<T, V>{});
    return;
  }
  T* state = (T*)a.state + slot * (K - 1) * a.channels + c;
  Pack<T, V> row[K];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) row[i] = load_pack<T, V>(state + (int64_t)i * a.channels);
  row[K - 1] = load_pack<T, V>((const T*)a.x + n * a.x_row + c);
  const ConvWeight<T, V, K> w(a.weight, a.bias, c);
  constexpr int P = (V + 1) / 2;
  f32x2 o[P];
#pragma unroll
  for (int v = 0; v < P; ++v) o[v] = w.bias[v];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    f32x2 f[P];
    to_pairs<T, V>(row[k], f);
#pragma unroll
    for (int v = 0; v < P; ++v) o[v] = fma2(w.w[k][v], f[v], o[v]);
    if (k) store_pack<T, V>(state + (int64_t)(k - 1) * a.channels, row[k]);
  }
#pragma unroll
  for (int v = 0; v < P; ++v) o[v] = a.silu ? mul2(o[v], sigmoid(o[v])) : o[v];
  store_pack<T, V>(to, from_pairs<T, V>(o));
}

template <class T, int V, int K>
cudaError_t go(const ConvLaunch& l, cudaStream_t s) {
  const int64_t per_y = l.threads / l.per_x, rows = l.runs + (l.a.state_out ? l.a.grids : 0);
  k_conv<T, V, K><<<(unsigned)((rows + per_y - 1) / per_y * l.blocks_x), l.threads, 0, s>>>(l);
  return cudaGetLastError();
}
template <class T, int V, int K>
cudaError_t go(const ConvBackwardLaunch& l, cudaStream_t s) {
  const int64_t per_y = l.f.threads / l.f.per_x, more = l.g.dstate ? (l.f.a.grids + per_y - 1) / per_y : 0;
  if (l.parts + more)
    k_conv_backward<T, V, K><<<(unsigned)((l.parts + more) * l.f.blocks_x), l.f.threads, 0, s>>>(l);
  return cudaGetLastError();
}
template <class T, int V, int K>
cudaError_t go(const ConvStepLaunch& l, cudaStream_t s) {
  const int64_t n = l.a.streams * (l.a.channels / V);
  k_conv_step<T, V, K><<<(unsigned)((n + kConvThreads - 1) / kConvThreads), kConvThreads, 0, s>>>(l);
  return cudaGetLastError();
}
template <class T, int V, class L>
cudaError_t by_taps(const L& l, int taps, cudaStream_t s) {
  return taps == 2 ? go<T, V, 2>(l, s) : taps == 3 ? go<T, V, 3>(l, s) : go<T, V, 4>(l, s);
}
// Vectors of `bytes`, or single elements.
template <int bytes, class L>
cudaError_t by_type(const L& l, int type, int vec, int taps, cudaStream_t s) {
  switch (type) {
    case TB_TYPE_F32: return vec > 1 ? by_taps<float, bytes / 4>(l, taps, s) : by_taps<float, 1>(l, taps, s);
    case TB_TYPE_F16: return vec > 1 ? by_taps<__half, bytes / 2>(l, taps, s) : by_taps<__half, 1>(l, taps, s);
    default: return vec > 1 ? by_taps<__nv_bfloat16, bytes / 2>(l, taps, s) : by_taps<__nv_bfloat16, 1>(l, taps, s);
  }
}

}  // namespace

cudaError_t launch_conv(const void* args, cudaStream_t s) {
  const ConvLaunch& l = *(const ConvLaunch*)args;
  return by_type<16>(l, l.a.type, l.vec, l.a.taps, s);
}
cudaError_t launch_conv_backward(const void* args, cudaStream_t s) {
  const ConvBackwardLaunch& l = *(const ConvBackwardLaunch*)args;
  return by_type<8>(l, l.f.a.type, l.f.vec, l.f.a.taps, s);
}
cudaError_t launch_conv_weight(const void* args, cudaStream_t s) {
  const ConvBackwardLaunch& l = *(const ConvBackwardLaunch*)args;
  const unsigned blocks = (unsigned)(((int64_t)(l.f.a.taps + 1) * l.f.a.channels + 31) / 32);
  auto go = [&](auto kernel) { return launch_early(kernel, blocks, 512, 0, s, l.f.a.tokens > 0, l); };
  switch (l.f.a.type) {
    case TB_TYPE_F32: return go(k_conv_weight<float>);
    case TB_TYPE_F16: return go(k_conv_weight<__half>);
    default: return go(k_conv_weight<__nv_bfloat16>);
  }
}
cudaError_t launch_conv_step(const void* args, cudaStream_t s) {
  const ConvStepLaunch& l = *(const ConvStepLaunch*)args;
  return by_type<16>(l, l.a.type, l.vec, l.a.taps, s);
}

}  // namespace tb
