// Selective scan: the walk over rows, the joining of segments and the step for
// single tokens (tb_selective_scan, tb_selective_scan_step).
//
//   h_t = exp(delta_t a) h_(t-1) + delta_t x_t b_t,  y_t = (c_t . h_t + d x_t) silu(z_t)
//
// The states stay in registers (tb_scan.cuh); rows come through shared memory,
// eight at a time, the next ones on their way while eight are walked.  A call
// with few grids and channels is split along the rows: the segments' own last
// states first (from zero), their joining, then the outputs.  A segment's decay
// as a whole is exp(a sum of delta), so joining needs the sum alone.
#include "tb_scan.cuh"

namespace tb {
namespace {

constexpr int kWarps = 4;  // of a block: neighbouring channels of the same rows

// One warp's shared memory.
template <class T, int NN, bool kOut>
struct alignas(16) WalkShared {
  T raw[2][kOut ? 3 : 2][kScanRows][kScanChannels];  // x, dt, z of two tiles
  float delta[kScanRows][kScanChannels], dx[kScanRows][kScanChannels];
  float b[kScanRows][4 * NN], c[kOut ? kScanRows : 1][4 * NN];
  float part[kOut ? kScanRows : 1][4][kScanChannels];  // c . h over a lane's states
};

// kOut: the outputs from the states that the segments start from; else the
// segments' own states from zero and their sums of delta.  kMany: more states
// than a pass takes; those of a tile wait in shared memory (h, after the warps'
// own part) while the others' pass.
template <class T, int NN, bool kOut, bool kMany>
__global__ void __launch_bounds__(32 * kWarps) k_scan(ScanLaunch l) {
  extern __shared__ __align__(16) char s_raw[];
  typedef WalkShared<T, NN, kOut> Shared;
  if (kOut) wait_for_last_kernel();
  let_next_kernel_start();
  const tb_scan_args& a = l.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Shared& s = reinterpret_cast<Shared*>(s_raw)[warp];
  const int blocks = l.pad / (4 * NN);  // of states
  float* s_h = reinterpret_cast<float*>(s_raw + kWarps * sizeof(Shared)) + (int64_t)warp * blocks * 16 * NN * 8;
  const int slot = (int)(blockIdx.x / l.blocks_x), at = (int)(blockIdx.x % l.blocks_x) * kWarps + warp;
  const ScanTile t = scan_tile(l, at / l.group_tiles, at % l.group_tiles);
  if (t.group >= a.groups) return;
  const LinSegment seg = lin_segment(l, slot);
  if (kOut) scan_zero_share<T>(l, a.y, a.y_row, slot, t);
  if (seg.grid < 0 || (!kOut && seg.index + 1 == seg.count)) return;  // the last segment's own state joins no other
  const int64_t row0 = seg.begin + seg.first, state_at = (int64_t)seg.grid * a.channels * a.states;
  float* const own = l.seg + (int64_t)slot * a.channels * l.pad;
  float h[4][NN], a2[4][NN];
  auto load_a = [&](int n0) {
    read_dense<NN>(a2, a.a, t, a.states, n0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int n = 0; n < NN; ++n) a2[i][n] *= kLog2e;
  };
  auto first = [&](int n0) {
    if (kOut && l.segment) read_pad<NN>(h, own, t, l.pad, n0);
    else read_dense<NN>(h, kOut && a.state ? a.state + state_at : nullptr, t, a.states, n0);
  };
  auto kept = [&](int k) { return reinterpret_cast<float4*>(s_h + k * 16 * NN * 8) + lane; };  // NN vectors, 32 apart
  auto put = [&](int k) {
#pragma unroll
    for (int n = 0; n < NN; ++n) kept(k)[32 * n] = make_float4(h[0][n], h[1][n], h[2][n], h[3][n]);
  };
  auto get = [&](int k) {
#pragma unroll
    for (int n = 0; n < NN; ++n) {
      const float4 v = kept(k)[32 * n];
      h[0][n] = v.x, h[1][n] = v.y, h[2][n] = v.z, h[3][n] = v.w;
    }
  };
  if (kMany) {
    for (int k = 0; k < blocks; ++k) {
      first(k * 4 * NN);
      put(k);
    }
  } else {
    load_a(0);
    first(0);
  }
  const bool here = lane < t.count;
  const float bias = here && a.dt_bias ? a.dt_bias[t.first + lane] : 0.f;
  const float skip = kOut && here && a.d ? a.d[t.first + lane] : 0.f;
  const int tiles = (seg.len + kScanRows - 1) / kScanRows;
  auto fetch = [&](int i) {
    const int n = min(kScanRows, seg.len - i * kScanRows);
    if (n > 0) {
      const int64_t row = row0 + (int64_t)i * kScanRows;
      auto& raw = s.raw[i & 1];
      scan_fetch<T>(&raw[0][0][0], a.x, a.x_row, row, n, t, l.vec);
      scan_fetch<T>(&raw[1][0][0], a.dt, a.dt_row, row, n, t, l.vec);
      if constexpr (kOut)
        if (a.z) scan_fetch<T>(&raw[2][0][0], a.z, a.z_row, row, n, t, l.vec);
    }
    scan_fetched();
  };
  ScanStates<T, NN> nb, nc;
  auto load_states = [&](int i, int n0) {
    const int64_t row = row0 + (int64_t)i * kScanRows;
    const int n = min(kScanRows, seg.len - i * kScanRows);
    nb.load(a.b, a.b_row, t.group * a.b_group, row, n, a.states, n0);
    if (kOut) nc.load(a.c, a.c_row, t.group * a.c_group, row, n, a.states, n0);
  };
  const int c4 = lane / 4 * 4, s4 = lane % 4 * NN;
  float total = 0.f;
  fetch(0);
  load_states(0, 0);
  for (int i = 0; i < tiles; ++i) {
    const int n = min(kScanRows, seg.len - i * kScanRows);
    fetch(i + 1);
    scan_wait<1>();
    auto& raw = s.raw[i & 1];
#pragma unroll
    for (int r = 0; r < kScanRows; ++r) {
      const float v = RowType<T>::to(raw[1][r][lane]) + bias;
      const float delta = r < n ? (a.softplus ? scan_softplus(v) : v) : 0.f;
      total += delta;
      s.delta[r][lane] = delta;
      s.dx[r][lane] = delta * RowType<T>::to(raw[0][r][lane]);
    }
    for (int k = 0; k < (kMany ? blocks : 1); ++k) {
      nb.store(&s.b[0][0]);
      if (kOut) nc.store(&s.c[0][0]);
      __syncwarp();
      if (kMany) {
        load_a(k * 4 * NN);
        get(k);
        if (k + 1 < blocks) load_states(i, (k + 1) * 4 * NN);
        else load_states(i + 1, 0);
      } else {
        load_states(i + 1, 0);
      }
#pragma unroll
      for (int r = 0; r < kScanRows; ++r) {
        float d[4], x[4], b[NN], c[NN], y[4] = {};
        read_channels(d, &s.delta[r][c4]);
        read_channels(x, &s.dx[r][c4]);
        read_states<NN>(b, &s.b[r][s4]);
        if (kOut) read_states<NN>(c, &s.c[r][s4]);
#pragma unroll
        for (int n = 0; n < NN; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            h[j][n] = fmaf(scan_decay(d[j], a2[j][n]), h[j][n], x[j] * b[n]);
            if (kOut) y[j] = fmaf(c[n], h[j][n], y[j]);
          }
        if constexpr (kOut) {
          float* to = &s.part[r][lane % 4][c4];
          if (kMany && k) {
            float f[4];
            read_channels(f, to);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] += f[j];
          }
          write_channels(to, y);
        }
      }
      if (kMany) put(k);
      __syncwarp();
    }
    if constexpr (kOut) {
      T* to = (T*)a.y + (row0 + (int64_t)i * kScanRows) * a.y_row + t.first + lane;
#pragma unroll
      for (int r = 0; r < kScanRows; ++r) {
        float y = (s.part[r][0][lane] + s.part[r][1][lane]) + (s.part[r][2][lane] + s.part[r][3][lane]);
        y = fmaf(skip, RowType<T>::to(raw[0][r][lane]), y);
        if (a.z) {
          const float z = RowType<T>::to(raw[2][r][lane]);
          y *= z * scan_sigmoid(z);
        }
        if (here && r < n) to[r * a.y_row] = RowType<T>::from(y);
      }
      __syncwarp();
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  for (int k = 0; k < (kMany ? blocks : 1); ++k) {
    if (kMany) get(k);
    if (!kOut) write_pad<NN>(own, h, t, l.pad, k * 4 * NN);
    else if (a.state_out && seg.index + 1 == seg.count) write_dense<NN>(a.state_out + state_at, h, t, a.states, k * 4 * NN);
  }
  if (!kOut && here) l.sum[(int64_t)slot * a.channels + t.first + lane] = total;
}

// Joins the segments: the state that each one starts from, in place of its own.
// A thread takes four states of a channel of a grid.
constexpr int kJoinBatch = 8;
__global__ void __launch_bounds__(128) k_scan_join(ScanLaunch l) {
  let_next_kernel_start();
  const tb_scan_args& a = l.a;
  const int per = l.pad / 4, blocks = (int)(((int64_t)a.channels * per + blockDim.x - 1) / blockDim.x);
  const int b = blockIdx.x / blocks, slot0 = lin_first_slot(l, b);
  int64_t begin, end;
  lin_grid_rows(l, b, begin, end);
  // offsets that decrease name rows twice: their segments are more than the slots, which bound the walk
  const int n = min(lin_segments_of(l, end - begin), max(0, l.segments - slot0));
  const int64_t i = (int64_t)(blockIdx.x % blocks) * blockDim.x + threadIdx.x, c = i / per;
  if (c >= a.channels) return;
  const int s = (int)(i - c * per) * 4;
  float a2[4], x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool is = s + k < a.states;
    a2[k] = is ? a.a[c * a.states + s + k] * kLog2e : 0.f;
    x[k] = is && a.state ? a.state[((int64_t)b * a.channels + c) * a.states + s + k] : 0.f;
  }
  wait_for_last_kernel();
  float* at = l.seg + ((int64_t)slot0 * a.channels + c) * l.pad + s;
  const float* sum = l.sum + (int64_t)slot0 * a.channels + c;
  const int64_t next = (int64_t)a.channels * l.pad;
  for (int j0 = 0; j0 < n; j0 += kJoinBatch) {
    float4 own[kJoinBatch];
    float d[kJoinBatch];
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j)
      if (j0 + j + 1 < n) {
        own[j] = *reinterpret_cast<const float4*>(at + (j0 + j) * next);
        d[j] = sum[(int64_t)(j0 + j) * a.channels];
      }
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j)
      if (j0 + j < n) {
        *reinterpret_cast<float4*>(at + (j0 + j) * next) = make_float4(x[0], x[1], x[2], x[3]);
        if (j0 + j + 1 < n) {
          const float f[4] = {own[j].x, own[j].y, own[j].z, own[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = fmaf(scan_decay(d[j], a2[k]), x[k], f[k]);
        }
      }
  }
}

// ---------------------------------------------------------------- one token
//
// 8 bytes a state and nothing else of size: the bound is memory.  Four lanes
// take a channel, V states at a time each.
template <class T, int V>
__global__ void __launch_bounds__(128) k_scan_step(ScanStepLaunch l) {
  const tb_scan_step_args& a = l.a;
  const int64_t n = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  const int c = (int)(blockIdx.x * 32 + threadIdx.x / 4), lane = threadIdx.x % 4;
  if (n >= a.streams) return;
  const bool live = c < a.channels;
  const int64_t slot = a.slots ? (int64_t)a.slots[n] : n;
  T* to = (T*)a.y + n * a.y_row + c;
  if (slot < 0 || slot >= a.num_slots) {
    if (live && lane == 0) *to = RowType<T>::from(0.f);
    return;
  }
  float sum = 0.f, x = 0.f;
  if (live) {
    const int group = c / (a.channels / a.groups);
    float* h = a.state + (slot * a.channels + c) * (int64_t)a.states;
    const float* rate = a.a + (int64_t)c * a.states;
    const T* b = (const T*)a.b + n * a.b_row + group * a.b_group;
    const T* cc = (const T*)a.c + n * a.c_row + group * a.c_group;
    x = RowType<T>::to(((const T*)a.x)[n * a.x_row + c]);
    float delta = RowType<T>::to(((const T*)a.dt)[n * a.dt_row + c]) + (a.dt_bias ? a.dt_bias[c] : 0.f);
    if (a.softplus) delta = scan_softplus(delta);
    const float dx = delta * x;
    for (int s = lane * V; s < a.states; s += 4 * V) {
      float f[V], r[V];
      unpack<float, V>(load_pack<float, V>(h + s), f);
#pragma unroll
      for (int k = 0; k < V; ++k) r[k] = rate[s + k];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        f[k] = fmaf(scan_decay(delta, r[k] * kLog2e), f[k], dx * RowType<T>::to(b[s + k]));
        sum = fmaf(RowType<T>::to(cc[s + k]), f[k], sum);
      }
      store_pack<float, V>(h + s, pack<float, V>(f));
    }
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  if (live && lane == 0) {
    float y = a.d ? fmaf(a.d[c], x, sum) : sum;
    if (a.z) {
      const float z = RowType<T>::to(((const T*)a.z)[n * a.z_row + c]);
      y *= z * scan_sigmoid(z);
    }
    *to = RowType<T>::from(y);
  }
}

template <class T, int NN, bool kOut, bool kMany>
cudaError_t go(const ScanLaunch& l, cudaStream_t s) {
  size_t bytes = kWarps * sizeof(WalkShared<T, NN, kOut>);
  if (kMany) bytes += (size_t)kWarps * (l.pad / (4 * NN)) * 16 * NN * 8 * sizeof(float);
  static std::atomic<bool> ready[kMaxDevices];
  const cudaError_t e = allow_shared(k_scan<T, NN, kOut, kMany>, 227 * 1024, ready);
  if (e != cudaSuccess) return e;
  return launch_early(k_scan<T, NN, kOut, kMany>, (unsigned)((int64_t)l.segments * l.blocks_x), 32 * kWarps, bytes, s,
                      kOut && l.segment != 0, l);
}
template <class T, bool kOut>
cudaError_t pick(const ScanLaunch& l, cudaStream_t s) {
  if (l.nn == 2) return go<T, 2, kOut, false>(l, s);
  return l.pad == 16 ? go<T, 4, kOut, false>(l, s) : go<T, 4, kOut, true>(l, s);
}
template <bool kOut>
cudaError_t by_type(const ScanLaunch& l, cudaStream_t s) {
  switch (l.a.type) {
    case TB_TYPE_F32: return pick<float, kOut>(l, s);
    case TB_TYPE_F16: return pick<__half, kOut>(l, s);
    default: return pick<__nv_bfloat16, kOut>(l, s);
  }
}

}  // namespace

cudaError_t launch_scan(const void* args, cudaStream_t s) { return by_type<true>(*(const ScanLaunch*)args, s); }
cudaError_t launch_scan_states(const void* args, cudaStream_t s) { return by_type<false>(*(const ScanLaunch*)args, s); }

cudaError_t launch_scan_join(const void* args, cudaStream_t s) {
  const ScanLaunch& l = *(const ScanLaunch*)args;
  const int64_t items = (int64_t)l.a.channels * (l.pad / 4);
  return launch_early(k_scan_join, (unsigned)((items + 127) / 128 * l.grids), 128, 0, s, true, l);
}

cudaError_t launch_scan_step(const void* args, cudaStream_t s) {
  const ScanStepLaunch& l = *(const ScanStepLaunch*)args;
  const unsigned y = (unsigned)(l.a.streams < 32768 ? l.a.streams : 32768);
  const dim3 grid((l.a.channels + 31) / 32, y, (unsigned)((l.a.streams + y - 1) / y));
  auto go = [&](auto four, auto one) {
    if (l.a.states % 4 == 0) four<<<grid, 128, 0, s>>>(l);
    else one<<<grid, 128, 0, s>>>(l);
    return cudaGetLastError();
  };
  switch (l.a.type) {
    case TB_TYPE_F32: return go(k_scan_step<float, 4>, k_scan_step<float, 1>);
    case TB_TYPE_F16: return go(k_scan_step<__half, 4>, k_scan_step<__half, 1>);
    default: return go(k_scan_step<__nv_bfloat16, 4>, k_scan_step<__nv_bfloat16, 1>);
  }
}

}  // namespace tb
