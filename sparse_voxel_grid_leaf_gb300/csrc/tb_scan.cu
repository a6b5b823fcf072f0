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
  Two b[kScanRows][4 * NN], c[kOut ? kScanRows : 1][4 * NN];
  float part[kOut ? kScanRows : 1][4][kScanChannels];  // c . h over a lane's states
};

// kOut: the outputs from the states that the segments start from; else the
// segments' own states from zero and their sums of delta.  kMany: more states
// than a pass takes; those of a tile wait in shared memory (after the warps'
// own part) while the others' pass.
template <class T, int NN, bool kOut, bool kMany>
__global__ void __launch_bounds__(32 * kWarps) k_scan(ScanLaunch l) {
  extern __shared__ __align__(16) char s_raw[];
  typedef WalkShared<T, NN, kOut> Shared;
  if (kOut) wait_for_last_kernel();
  let_next_kernel_start();
  const tb_scan_args& a = l.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, o = lane >> 4;
  Shared& s = reinterpret_cast<Shared*>(s_raw)[warp];
  const int blocks = kMany ? l.pad / (4 * NN) : 1;  // of states
  float* s_h = reinterpret_cast<float*>(s_raw + kWarps * sizeof(Shared)) + (int64_t)warp * blocks * 128 * NN;
  const int slot = (int)(blockIdx.x / l.blocks_x), at = (int)(blockIdx.x % l.blocks_x) * kWarps + warp;
  const ScanTile t = scan_tile(l, at / l.group_tiles, at % l.group_tiles);
  if (t.group >= a.groups) return;
  const LinSegment seg = lin_segment(l, slot);
  if (kOut) scan_zero_share<T>(l, a.y, a.y_row, slot, t);
  if (seg.grid < 0 || (!kOut && seg.index + 1 == seg.count)) return;  // the last segment's own state joins no other
  const int64_t row0 = seg.begin + seg.first, state_at = (int64_t)seg.grid * a.channels * a.states;
  float* const own = l.seg + (int64_t)slot * a.channels * l.pad;
  Two h[2][NN] = {}, a2[2][NN];
  auto first = [&](int n0) {
    if (kOut && l.segment) read_pad<NN>(h, own, t, l.pad, n0);
    else if (kOut) read_dense<NN>(h, a.state ? a.state + state_at : nullptr, t, a.states, n0);
  };
  if (kMany) {
    for (int k = 0; k < blocks; ++k) {
      first(k * 4 * NN);
      keep_states<NN>(s_h + k * 128 * NN, h);
    }
  } else {
    read_rates<NN>(a2, a, t, 0);
    first(0);
  }
  const Two bias = channel_pair(a.dt_bias, t), skip = channel_pair(kOut ? a.d : nullptr, t);
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
  ScanStates<T, NN> nb(a.b, a.b_row, t.group * a.b_group, row0, a.states, 0), nc(a.c, a.c_row, t.group * a.c_group, row0, a.states, 0);
  auto load_states = [&](int i, int n0) {
    const int n = min(kScanRows, seg.len - i * kScanRows);
    if (kMany) {
      nb = ScanStates<T, NN>(a.b, a.b_row, t.group * a.b_group, row0, a.states, n0);
      if (kOut) nc = ScanStates<T, NN>(a.c, a.c_row, t.group * a.c_group, row0, a.states, n0);
    }
    nb.load(i * kScanRows, n);
    if (kOut) nc.load(i * kScanRows, n);
  };
  PairOut<T> out(a.y, a.y_row, row0, t);
  const int c4 = lane / 4 * 4, s4 = lane % 4 * NN;
  Two total = 0;
  fetch(0);
  load_states(0, 0);
  for (int i = 0; i < tiles; ++i) {
    const int n = min(kScanRows, seg.len - i * kScanRows);
    fetch(i + 1);
    scan_wait<1>();
    auto& raw = s.raw[i & 1];
#pragma unroll
    for (int r = o; r < kScanRows; r += 2) {
      Two delta = scan_step_of(row_pair<T>(raw[1][r]), bias, a.softplus);
      if (r >= n) delta = 0;
      total = add2(total, delta);
      pair_of(s.delta[r]) = delta;
      pair_of(s.dx[r]) = mul2(delta, row_pair<T>(raw[0][r]));
    }
    for (int k = 0; k < blocks; ++k) {
      nb.store(s.b);
      if constexpr (kOut) nc.store(s.c);
      __syncwarp();
      if (kMany) {
        read_rates<NN>(a2, a, t, k * 4 * NN);
        kept_states<NN>(h, s_h + k * 128 * NN);
      }
      if (kMany && k + 1 < blocks) load_states(i, (k + 1) * 4 * NN);
      else load_states(i + 1, 0);
#pragma unroll
      for (int r = 0; r < kScanRows; ++r) {
        Two d[2], x[2], b[NN], c[NN], y[2] = {};
        read_pairs<2>(d, &s.delta[r][c4]);
        read_pairs<2>(x, &s.dx[r][c4]);
        read_pairs<NN>(b, &s.b[r][s4]);
        if constexpr (kOut) read_pairs<NN>(c, &s.c[r][s4]);
#pragma unroll
        for (int n = 0; n < NN; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            h[j][n] = fma2(scan_decay(d[j], a2[j][n]), h[j][n], mul2(x[j], b[n]));
            if (kOut) y[j] = n ? fma2(c[n], h[j][n], y[j]) : mul2(c[n], h[j][n]);
          }
        if constexpr (kOut) {
          float* to = &s.part[r][lane % 4][c4];
          if (kMany && k) {
            Two f[2];
            read_pairs<2>(f, to);
            y[0] = add2(y[0], f[0]), y[1] = add2(y[1], f[1]);
          }
          write_pairs(to, y);
        }
      }
      if (kMany) keep_states<NN>(s_h + k * 128 * NN, h);
      __syncwarp();
    }
    if constexpr (kOut) {
#pragma unroll
      for (int r = o; r < kScanRows; r += 2) {
        Two y = add2(add2(pair_of(s.part[r][0]), pair_of(s.part[r][1])), add2(pair_of(s.part[r][2]), pair_of(s.part[r][3])));
        y = fma2(skip, row_pair<T>(raw[0][r]), y);
        if (a.z) {
          const Two z = row_pair<T>(raw[2][r]);
          y = mul2(y, mul2(z, scan_sigmoid(z)));
        }
        if (r < n) out.put(r, y);
      }
      out.at += kScanRows * out.stride;
      __syncwarp();
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  for (int k = 0; k < blocks; ++k) {
    if (kMany) kept_states<NN>(h, s_h + k * 128 * NN);
    if (!kOut) write_pad<NN>(own, h, t, l.pad, k * 4 * NN);
    else if (a.state_out && seg.index + 1 == seg.count) write_dense<NN>(a.state_out + state_at, h, t, a.states, k * 4 * NN);
  }
  if (!kOut) scan_put_sum(l, slot, t, total);
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
  if (kMany) bytes += (size_t)kWarps * (l.pad / (4 * NN)) * 128 * NN * sizeof(float);
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
