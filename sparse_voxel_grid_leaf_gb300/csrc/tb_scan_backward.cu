// The gradient of the selective scan (tb_selective_scan_backward).
//
// With ds = dy silu(z), s_t = c_t . h_t + d x_t and
//   g_t = c_t ds_t + exp(delta_(t+1) a) g_(t+1)
// per channel and state:
//   db_t = sum over channels g delta x,  dc_t = sum over channels ds h,
//   into = g . b,  dx = d ds + delta into,  q = g exp(delta a) h_(t-1),
//   ddelta = a . q + x into,  da = sum over rows q delta,  dz = dy s silu'(z).
//
// The rows are taken in chunks of kScanChunk.  First every chunk's own last
// state and its own part of the carried exp(delta a) g, both from zero, and
// their joining along the grids, forward and backward; then all chunks at once,
// each with what enters it from both sides.  A warp walks its chunk forward,
// keeping the state before every eighth row in shared memory, and then
// backward, four rows at a time with their states and decays in registers.
// Sums over channels go through shared memory over a block's four warps, and
// over blocks through parts that a last kernel adds in a fixed order.
#include "tb_scan.cuh"

namespace tb {
namespace {

constexpr int kWarps = 4;
constexpr int kTiles = kScanChunk / kScanRows;

// ------------------------------------------------- what the chunks carry back

template <class T, int NN>
struct alignas(16) CarryShared {
  T raw[2][3][kScanRows][kScanChannels];  // dt, dy, z of two tiles
  float delta[kScanRows][kScanChannels], ds[kScanRows][kScanChannels];
  Two c[kScanRows][4 * NN];
};

// One block of states a warp (blockIdx.y), as the walks are short.
template <class T, int NN>
__global__ void __launch_bounds__(32 * kWarps) k_scan_carry(ScanBackwardLaunch g) {
  extern __shared__ __align__(16) char s_raw[];
  let_next_kernel_start();
  const ScanLaunch& l = g.f;
  const tb_scan_args& a = l.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, o = lane >> 4;
  CarryShared<T, NN>& s = reinterpret_cast<CarryShared<T, NN>*>(s_raw)[warp];
  const int slot = (int)(blockIdx.x / l.blocks_x), at = (int)(blockIdx.x % l.blocks_x) * kWarps + warp;
  const int n0 = blockIdx.y * 4 * NN;
  const ScanTile t = scan_tile(l, at / l.group_tiles, at % l.group_tiles);
  if (t.group >= a.groups) return;
  const LinSegment seg = lin_segment(l, slot);
  if (seg.grid < 0 || (seg.index == 0 && !g.g.dstate)) return;  // the first chunk's goes nowhere else
  const int64_t row0 = seg.begin + seg.first;
  Two h[2][NN] = {}, a2[2][NN], total = 0;
  read_rates<NN>(a2, a, t, n0);
  const Two bias = channel_pair(a.dt_bias, t);
  const int tiles = (seg.len + kScanRows - 1) / kScanRows;
  auto fetch = [&](int i) {
    if (i >= 0) {
      const int n = min(kScanRows, seg.len - i * kScanRows);
      const int64_t row = row0 + i * kScanRows;
      auto& raw = s.raw[i & 1];
      scan_fetch<T>(&raw[0][0][0], a.dt, a.dt_row, row, n, t, l.vec);
      scan_fetch<T>(&raw[1][0][0], g.g.dy, g.g.dy_row, row, n, t, l.vec);
      if (a.z) scan_fetch<T>(&raw[2][0][0], a.z, a.z_row, row, n, t, l.vec);
    }
    scan_fetched();
  };
  ScanStates<T, NN> nc(a.c, a.c_row, t.group * a.c_group, row0, a.states, n0);
  auto load_states = [&](int i) { nc.load(i * kScanRows, i < 0 ? 0 : min(kScanRows, seg.len - i * kScanRows)); };
  const int c4 = lane / 4 * 4, s4 = lane % 4 * NN;
  fetch(tiles - 1);
  load_states(tiles - 1);
  for (int i = tiles - 1; i >= 0; --i) {
    const int n = min(kScanRows, seg.len - i * kScanRows);
    fetch(i - 1);
    scan_wait<1>();
    auto& raw = s.raw[i & 1];
#pragma unroll
    for (int r = o; r < kScanRows; r += 2) {
      Two ds = row_pair<T>(raw[1][r]);
      if (a.z) {
        const Two z = row_pair<T>(raw[2][r]);
        ds = mul2(ds, mul2(z, scan_sigmoid(z)));
      }
      Two delta = scan_step_of(row_pair<T>(raw[0][r]), bias, a.softplus);
      if (r >= n) delta = ds = 0;
      total = add2(total, delta);
      pair_of(s.delta[r]) = delta;
      pair_of(s.ds[r]) = ds;
    }
    nc.store(s.c);
    __syncwarp();
    load_states(i - 1);
#pragma unroll
    for (int r = kScanRows - 1; r >= 0; --r) {
      Two d[2], ds[2], c[NN];
      read_pairs<2>(d, &s.delta[r][c4]);
      read_pairs<2>(ds, &s.ds[r][c4]);
      read_pairs<NN>(c, &s.c[r][s4]);
#pragma unroll
      for (int n = 0; n < NN; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) h[j][n] = mul2(scan_decay(d[j], a2[j][n]), fma2(c[n], ds[j], h[j][n]));
    }
    __syncwarp();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  write_pad<NN>(g.seg_back + (int64_t)slot * a.channels * l.pad, h, t, l.pad, n0);
  if (blockIdx.y == 0) scan_put_sum(l, slot, t, total);  // a grid's last chunk has none yet
}

// Joins what the chunks carry back, from a grid's last chunk to its first: what
// enters each from behind, in place of its own, and the gradient of the first
// state.  A thread takes four states of a channel of a grid.
constexpr int kJoinBatch = 8;
__global__ void __launch_bounds__(128) k_scan_join_back(ScanBackwardLaunch g) {
  let_next_kernel_start();
  const ScanLaunch& l = g.f;
  const tb_scan_args& a = l.a;
  const int per = l.pad / 4, blocks = (int)(((int64_t)a.channels * per + blockDim.x - 1) / blockDim.x);
  const int b = blockIdx.x / blocks, slot0 = lin_first_slot(l, b);
  int64_t begin, end;
  lin_grid_rows(l, b, begin, end);
  const int n = min(lin_segments_of(l, end - begin), max(0, l.segments - slot0));
  const int64_t i = (int64_t)(blockIdx.x % blocks) * blockDim.x + threadIdx.x, c = i / per;
  if (c >= a.channels) return;
  const int s = (int)(i - c * per) * 4;
  const int64_t state_at = ((int64_t)b * a.channels + c) * a.states + s;
  float a2[4], x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool is = s + k < a.states;
    a2[k] = is ? a.a[c * a.states + s + k] * kLog2e : 0.f;
    x[k] = is && g.g.dstate_out ? g.g.dstate_out[state_at + k] : 0.f;
  }
  wait_for_last_kernel();
  float* at = g.seg_back + ((int64_t)slot0 * a.channels + c) * l.pad + s;
  const float* sum = l.sum + (int64_t)slot0 * a.channels + c;
  const int64_t next = (int64_t)a.channels * l.pad;
  const int least = g.g.dstate ? 0 : 1;  // the first chunk's own is made where the gradient is asked for
  for (int j0 = n - 1; j0 >= 0; j0 -= kJoinBatch) {
    float4 own[kJoinBatch];
    float d[kJoinBatch];
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j)
      if (j0 - j >= least) {
        own[j] = *reinterpret_cast<const float4*>(at + (j0 - j) * next);
        d[j] = sum[(int64_t)(j0 - j) * a.channels];
      }
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j)
      if (j0 - j >= 0) {
        *reinterpret_cast<float4*>(at + (j0 - j) * next) = make_float4(x[0], x[1], x[2], x[3]);
        if (j0 - j >= least) {
          const float f[4] = {own[j].x, own[j].y, own[j].z, own[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = fmaf(scan_decay(d[j], a2[k]), x[k], f[k]);
        }
      }
  }
  if (g.g.dstate)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s + k < a.states) g.g.dstate[state_at + k] = x[k];
}

// ------------------------------------------------------------ all of a chunk

template <class T, int NN>
struct alignas(16) BackShared {
  float kept[kTiles - 1][128 * NN];  // the states before the tiles but the first
  float delta[kScanRows][kScanChannels], dx[kScanRows][kScanChannels], ds[kScanRows][kScanChannels];
  Two b[kScanRows][4 * NN], c[kScanRows][4 * NN];
  float sums[2][3][4][kScanChannels];  // of two rows: a lane's c . h, g . b, a . q
  float bc[2][2][36 * NN];             // of two rows: a lane's channels of db, dc; on different banks
  T raw[4][kScanRows][kScanChannels];  // x, dt, z, dy
};

template <class T, int NN, bool kMany>
__global__ void __launch_bounds__(32 * kWarps, 2) k_scan_backward(ScanBackwardLaunch g) {
  extern __shared__ __align__(16) char s_raw[];
  typedef BackShared<T, NN> Shared;
  constexpr int kStates = 4 * NN;
  wait_for_last_kernel();
  let_next_kernel_start();
  const ScanLaunch& l = g.f;
  const tb_scan_args& a = l.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, o = lane >> 4, p = lane & 15;
  Shared& s = reinterpret_cast<Shared*>(s_raw)[warp];
  Two(*s_bc)[kScanRows][kStates] = reinterpret_cast<Two(*)[kScanRows][kStates]>(s_raw + kWarps * sizeof(Shared));
  const int per_run = a.groups * g.quads, run = (int)(blockIdx.x / per_run), at = (int)(blockIdx.x % per_run);
  const int group = at / g.quads, quad = at % g.quads;
  const ScanTile t = scan_tile(l, group, quad * kWarps + warp);
  const int c4 = lane / 4 * 4, s4 = lane % 4 * NN;
  const Two bias = channel_pair(a.dt_bias, t), skip = channel_pair(a.d, t);
  Two sum_d = 0, sum_bias = 0;
  const int blocks = kMany ? l.pad / kStates : 1;
  for (int k = 0; k < blocks; ++k) {
    const int n0 = k * kStates;
    const bool last = k + 1 == blocks;
    Two a2[2][NN], da[2][NN] = {};
    read_rates<NN>(a2, a, t, n0);
    for (int slot = run * g.per_run; slot < min((run + 1) * g.per_run, l.segments); ++slot) {
      if (k == 0) {
        scan_zero_share<T>(l, g.g.dx, g.g.dx_row, slot, t);
        scan_zero_share<T>(l, g.g.ddt, g.g.ddt_row, slot, t);
        if (a.z) scan_zero_share<T>(l, g.g.dz, g.g.dz_row, slot, t);
      }
      const LinSegment seg = lin_segment(l, slot);
      if (seg.grid < 0 || seg.len == 0) continue;
      const int64_t row0 = seg.begin + seg.first, own = (int64_t)slot * a.channels * l.pad;
      const int tiles = (seg.len + kScanRows - 1) / kScanRows;
      const PairOut<T> out_x(g.g.dx, g.g.dx_row, row0, t), out_dt(g.g.ddt, g.g.ddt_row, row0, t), out_z(g.g.dz, g.g.dz_row, row0, t);
      ScanStates<T, NN> nb(a.b, a.b_row, t.group * a.b_group, row0, a.states, n0), nc(a.c, a.c_row, t.group * a.c_group, row0, a.states, n0);
      Two h[2][NN];
      auto stage = [&](int i, bool all) {
        const int64_t row = row0 + i * kScanRows;
        const int n = min(kScanRows, seg.len - i * kScanRows);
        scan_fetch<T>(&s.raw[0][0][0], a.x, a.x_row, row, n, t, l.vec);
        scan_fetch<T>(&s.raw[1][0][0], a.dt, a.dt_row, row, n, t, l.vec);
        if (all) {
          if (a.z) scan_fetch<T>(&s.raw[2][0][0], a.z, a.z_row, row, n, t, l.vec);
          scan_fetch<T>(&s.raw[3][0][0], g.g.dy, g.g.dy_row, row, n, t, l.vec);
        }
        scan_fetched();
        nb.load(i * kScanRows, n);
        if (all) nc.load(i * kScanRows, n);
        nb.store(s.b);
        if (all) nc.store(s.c);
        scan_wait<0>();
#pragma unroll
        for (int r = o; r < kScanRows; r += 2) {
          Two delta = scan_step_of(row_pair<T>(s.raw[1][r]), bias, a.softplus);
          if (r >= n) delta = 0;
          pair_of(s.delta[r]) = delta;
          pair_of(s.dx[r]) = mul2(delta, row_pair<T>(s.raw[0][r]));
          if (all) {
            Two ds = row_pair<T>(s.raw[3][r]);
            if (a.z) {
              const Two z = row_pair<T>(s.raw[2][r]);
              ds = mul2(ds, mul2(z, scan_sigmoid(z)));
            }
            pair_of(s.ds[r]) = r < n ? ds : 0;
          }
        }
        __syncwarp();
      };
      auto forward = [&](int r, Two (&e)[2][NN]) {
        Two d[2], x[2], b[NN];
        read_pairs<2>(d, &s.delta[r][c4]);
        read_pairs<2>(x, &s.dx[r][c4]);
        read_pairs<NN>(b, &s.b[r][s4]);
#pragma unroll
        for (int n = 0; n < NN; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            e[j][n] = scan_decay(d[j], a2[j][n]);
            h[j][n] = fma2(e[j][n], h[j][n], mul2(x[j], b[n]));
          }
      };
      read_pad<NN>(h, l.seg + own, t, l.pad, n0);
      for (int i = 0; i + 1 < tiles; ++i) {
        stage(i, false);
#pragma unroll
        for (int r = 0; r < kScanRows; ++r) {
          Two e[2][NN];
          forward(r, e);
        }
        keep_states<NN>(s.kept[i], h);
        __syncwarp();
      }
      Two carry[2][NN];
      read_pad<NN>(carry, g.seg_back + own, t, l.pad, n0);
      for (int i = tiles - 1; i >= 0; --i) {
        const int rows = min(kScanRows, seg.len - i * kScanRows);
        stage(i, true);
#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
          if (i) kept_states<NN>(h, s.kept[i - 1]);
          else read_pad<NN>(h, l.seg + own, t, l.pad, n0);
          if (half) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              Two e[2][NN];
              forward(r, e);
            }
          }
          // the states before four rows and after each, and the rows' decays
          Two hs[5][2][NN], e[4][2][NN];
#pragma unroll
          for (int r = 0; r <= 4; ++r) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int n = 0; n < NN; ++n) hs[r][j][n] = h[j][n];
            if (r < 4) forward(4 * half + r, e[r]);
          }
#pragma unroll
          for (int r = 3; r >= 0; --r) {
            const int at_row = 4 * half + r;
            Two d[2], x[2], ds[2], b[NN], c[NN], y[2] = {}, into[2] = {}, qa[2] = {};
            float db[NN], dc[NN];
            read_pairs<2>(d, &s.delta[at_row][c4]);
            read_pairs<2>(x, &s.dx[at_row][c4]);
            read_pairs<2>(ds, &s.ds[at_row][c4]);
            read_pairs<NN>(b, &s.b[at_row][s4]);
            read_pairs<NN>(c, &s.c[at_row][s4]);
#pragma unroll
            for (int n = 0; n < NN; ++n) {
              Two sum_b = 0, sum_c = 0;
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const Two grad = fma2(c[n], ds[j], carry[j][n]);
                y[j] = n ? fma2(c[n], hs[r + 1][j][n], y[j]) : mul2(c[n], hs[r + 1][j][n]);
                sum_c = j ? fma2(ds[j], hs[r + 1][j][n], sum_c) : mul2(ds[j], hs[r + 1][j][n]);
                sum_b = j ? fma2(grad, x[j], sum_b) : mul2(grad, x[j]);
                into[j] = n ? fma2(grad, b[n], into[j]) : mul2(grad, b[n]);
                carry[j][n] = mul2(grad, e[r][j][n]);
                const Two q = mul2(carry[j][n], hs[r][j][n]);
                qa[j] = n ? fma2(q, a2[j][n], qa[j]) : mul2(q, a2[j][n]);
                da[j][n] = fma2(q, d[j], da[j][n]);
              }
              const float2 fb = parts(sum_b), fc = parts(sum_c);
              db[n] = fb.x + fb.y;
              dc[n] = fc.x + fc.y;
            }
            write_pairs(&s.sums[r & 1][0][lane % 4][c4], y);
            write_pairs(&s.sums[r & 1][1][lane % 4][c4], into);
            write_pairs(&s.sums[r & 1][2][lane % 4][c4], qa);
#pragma unroll
            for (int n = 0; n < NN; n += 2) {
              const int to = lane / 4 * kStates + s4 + n;
              *reinterpret_cast<float2*>(&s.bc[r & 1][0][to]) = make_float2(db[n], db[n + 1]);
              *reinterpret_cast<float2*>(&s.bc[r & 1][1][to]) = make_float2(dc[n], dc[n + 1]);
            }
            if (r & 1) continue;
            __syncwarp();
            // the sums of two rows, one each half of the warp: by channels, then by states of db and dc
            const int rr = at_row + o;
            Two sum[3];
#pragma unroll
            for (int v = 0; v < 3; ++v)
              sum[v] = add2(add2(pair_of(s.sums[o][v][0]), pair_of(s.sums[o][v][1])),
                            add2(pair_of(s.sums[o][v][2]), pair_of(s.sums[o][v][3])));
            const int to = i * kScanRows + rr;
            if (kMany && rr < rows) {
              float* acc = g.acc + ((row0 + to) * a.channels + t.first + 2 * p) * 3;
#pragma unroll
              for (int m = 0; m < 2; ++m)
                if (2 * p + m < t.count)
#pragma unroll
                  for (int v = 0; v < 3; ++v) {
                    float2 f = parts(sum[v]);
                    float& mine = m ? f.y : f.x;
                    if (k) mine += acc[3 * m + v];
                    if (!last) acc[3 * m + v] = mine;
                    sum[v] = two(f.x, f.y);
                  }
            }
            if (rr < rows && last) {
              const Two xf = row_pair<T>(s.raw[0][rr]), dsf = pair_of(s.ds[rr]);
              const Two inner = fma2(skip, xf, sum[0]);
              Two ddt = fma2(xf, sum[1], mul2(sum[2], both(kLn2)));
              if (a.softplus) ddt = mul2(ddt, scan_sigmoid(add2(row_pair<T>(s.raw[1][rr]), bias)));
              out_x.put(to, fma2(skip, dsf, mul2(pair_of(s.delta[rr]), sum[1])));
              out_dt.put(to, ddt);
              if (a.z) {
                const Two z = row_pair<T>(s.raw[2][rr]), sg = scan_sigmoid(z);
                const Two slope = mul2(sg, fma2(z, fma2(sg, both(-1.f), both(1.f)), both(1.f)));
                out_z.put(to, mul2(mul2(row_pair<T>(s.raw[3][rr]), inner), slope));
              }
              sum_d = fma2(dsf, xf, sum_d);
              sum_bias = add2(sum_bias, ddt);
            }
            if (p < kStates) {
              const Two* from = reinterpret_cast<const Two*>(&s.bc[o][p / (2 * NN)][0]) + p % (2 * NN);
              Two f = from[0];
#pragma unroll
              for (int m = 1; m < 8; ++m) f = add2(f, from[m * 2 * NN]);
              s_bc[warp][rr][p] = f;
            }
            __syncwarp();
          }
        }
        __syncthreads();
        if (threadIdx.x < kScanRows * kStates) {
          const int r = threadIdx.x / kStates, v = threadIdx.x % kStates;
          if (r < rows) {
            const Two f = add2(add2(s_bc[0][r][v], s_bc[1][r][v]), add2(s_bc[2][r][v], s_bc[3][r][v]));
            const int64_t row = ((int64_t)quad * l.tokens + row0 + i * kScanRows + r) * a.groups + group;
            *reinterpret_cast<Two*>(&g.bc[(row * 2 + v / (2 * NN)) * l.pad + n0 + v % (2 * NN) * 2]) = f;
          }
        }
        __syncthreads();
      }
    }
    write_pad<NN>(g.part_a + (int64_t)run * a.channels * l.pad, da, t, l.pad, n0);
  }
  sum_d = add2(sum_d, __shfl_xor_sync(0xffffffffu, sum_d, 16));
  sum_bias = add2(sum_bias, __shfl_xor_sync(0xffffffffu, sum_bias, 16));
  if (o == 0) {
    const float2 fd = parts(sum_d), fb = parts(sum_bias);
    float* to = g.part_d + (int64_t)run * 2 * a.channels + t.first + 2 * p;
    if (2 * p < t.count) to[0] = fd.x, to[a.channels] = fb.x;
    if (2 * p + 1 < t.count) to[1] = fd.y, to[a.channels + 1] = fb.y;
  }
}

// db and dc = the quads' parts summed, and da, dd, ddt_bias the runs', in fixed orders.
template <class T>
__global__ void __launch_bounds__(512) k_scan_sums(ScanBackwardLaunch g) {
  __shared__ float s[16][33];
  const ScanLaunch& l = g.f;
  const tb_scan_args& a = l.a;
  const int64_t elements = l.tokens * a.groups * 2 * a.states, rows_blocks = (elements + 511) / 512;
  wait_for_last_kernel();
  if (blockIdx.x < rows_blocks) {
    const int64_t i = (int64_t)blockIdx.x * 512 + threadIdx.x;
    if (i >= elements) return;
    const int n = (int)(i % a.states), which = (int)(i / a.states % 2);
    const int64_t rg = i / (2 * a.states), row = rg / a.groups;
    const LinCover cover = lin_cover(l);
    float sum = 0.f;
    if (row >= cover.begin && row < cover.end)
      for (int q = 0; q < g.quads; ++q) sum += g.bc[(((int64_t)q * l.tokens * a.groups + rg) * 2 + which) * l.pad + n];
    ((T*)(which ? g.g.dc : g.g.db))[rg * a.states + n] = RowType<T>::from(sum);
    return;
  }
  const int64_t per_a = (int64_t)a.channels * l.pad, width = per_a + 2 * (int64_t)a.channels;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t o = (blockIdx.x - rows_blocks) * 32 + x;
  float sum = 0.f;
  if (o < width) {
    const float* part = o < per_a ? g.part_a + o : g.part_d + (o - per_a);
    const int64_t stride = o < per_a ? per_a : 2 * (int64_t)a.channels;
    for (int r = y; r < g.runs; r += 16) sum += part[r * stride];
  }
  s[y][x] = sum;
  __syncthreads();
  if (y || o >= width) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) sum += s[i][x];
  if (o < per_a) {
    const int64_t c = o / l.pad;
    const int n = (int)(o - c * l.pad);
    if (n < a.states) g.g.da[c * a.states + n] = sum;
  } else if (o - per_a < a.channels) {
    if (g.g.dd) g.g.dd[o - per_a] = sum;
  } else if (g.g.ddt_bias) {
    g.g.ddt_bias[o - per_a - a.channels] = sum;
  }
}

template <class T, int NN>
cudaError_t go_carry(const ScanBackwardLaunch& g, cudaStream_t s) {
  static std::atomic<bool> ready[kMaxDevices];
  const int bytes = kWarps * sizeof(CarryShared<T, NN>);
  const cudaError_t e = allow_shared(k_scan_carry<T, NN>, bytes, ready);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((int64_t)g.f.segments * g.f.blocks_x), g.f.pad / (4 * NN));
  k_scan_carry<T, NN><<<grid, 32 * kWarps, bytes, s>>>(g);
  return cudaGetLastError();
}
template <class T, int NN, bool kMany>
cudaError_t go_back(const ScanBackwardLaunch& g, cudaStream_t s) {
  static std::atomic<bool> ready[kMaxDevices];
  const int bytes = kWarps * (sizeof(BackShared<T, NN>) + kScanRows * 8 * NN * sizeof(float));
  const cudaError_t e = allow_shared(k_scan_backward<T, NN, kMany>, bytes, ready);
  if (e != cudaSuccess) return e;
  return launch_early(k_scan_backward<T, NN, kMany>, (unsigned)((int64_t)g.runs * g.f.a.groups * g.quads), 32 * kWarps, bytes, s,
                      true, g);
}
template <class T>
cudaError_t back(const ScanBackwardLaunch& g, cudaStream_t s) {
  if (g.f.nn == 2) return go_back<T, 2, false>(g, s);
  return g.f.pad == 16 ? go_back<T, 4, false>(g, s) : go_back<T, 4, true>(g, s);
}
template <class T>
cudaError_t carry(const ScanBackwardLaunch& g, cudaStream_t s) {
  return g.f.nn == 2 ? go_carry<T, 2>(g, s) : go_carry<T, 4>(g, s);
}

}  // namespace

cudaError_t launch_scan_back_states(const void* args, cudaStream_t s) {
  const ScanBackwardLaunch& g = *(const ScanBackwardLaunch*)args;
  switch (g.f.a.type) {
    case TB_TYPE_F32: return carry<float>(g, s);
    case TB_TYPE_F16: return carry<__half>(g, s);
    default: return carry<__nv_bfloat16>(g, s);
  }
}
cudaError_t launch_scan_back_join(const void* args, cudaStream_t s) {
  const ScanBackwardLaunch& g = *(const ScanBackwardLaunch*)args;
  const int64_t items = (int64_t)g.f.a.channels * (g.f.pad / 4);
  return launch_early(k_scan_join_back, (unsigned)((items + 127) / 128 * g.f.grids), 128, 0, s, true, g);
}
cudaError_t launch_scan_backward(const void* args, cudaStream_t s) {
  const ScanBackwardLaunch& g = *(const ScanBackwardLaunch*)args;
  switch (g.f.a.type) {
    case TB_TYPE_F32: return back<float>(g, s);
    case TB_TYPE_F16: return back<__half>(g, s);
    default: return back<__nv_bfloat16>(g, s);
  }
}
cudaError_t launch_scan_sums(const void* args, cudaStream_t s) {
  const ScanBackwardLaunch& g = *(const ScanBackwardLaunch*)args;
  const tb_scan_args& a = g.f.a;
  const int64_t rows = (g.f.tokens * a.groups * 2 * a.states + 511) / 512;
  const int64_t columns = ((int64_t)a.channels * (g.f.pad + 2) + 31) / 32;
  auto go = [&](auto kernel) { return launch_early(kernel, (unsigned)(rows + columns), 512, 0, s, g.runs > 0, g); };
  switch (a.type) {
    case TB_TYPE_F32: return go(k_scan_sums<float>);
    case TB_TYPE_F16: return go(k_scan_sums<__half>);
    default: return go(k_scan_sums<__nv_bfloat16>);
  }
}

}  // namespace tb
