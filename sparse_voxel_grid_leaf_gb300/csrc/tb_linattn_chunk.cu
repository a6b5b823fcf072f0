// Linear attention with a decay for each head on the tensor cores: bfloat16
// rows, heads of up to 128 keys and values, in chunks of 64 rows.
//
// Over a chunk of n rows (i, j count the rows in the order of the walk) with
// entering state X, and with r = 31, e = 1 forward and 0 in reverse order:
//   W_j   = fold decay^(r-j) c_j
//   A_i   = sum_(j<=i) (a_i . b_j) W_j + a_i (decay^(r+e) X)
//   out_i = mul decay^(i-r) A_i
//   X'    = decay^n X + decay^(n-e-r) sum_j b_j W_j
// The powers belong to single rows, so the scores a_i . b_j are only masked,
// both parts of an output meet in one accumulator, and the state goes through
// the chunks as Z = decay^(r+e) X, the operand itself: Z' = decay^64 (Z + B^T W).
// Exponents run from -32 to 32, which 32 bits (and bfloat16) hold with room
// for the values where the decay is in [kSteep, 1 / kSteep]; heads outside
// that range forget within a few rows and take the recurrence.
//
// Four products a chunk, each with the values (or, for the scores, the rows i)
// along the 128 lanes of tensor memory:
//   A B^T                     both operands in shared memory    -> scores
//   Z^T A^T  +  W^T scores^T  left operands in tensor memory    -> A^T
//   W^T B                     left operand in tensor memory     -> (B^T W)^T
// so that the state Z^T stays in the registers of the threads of its lanes (a
// value each), in 32 bits, and is rounded only as an operand.
//
// Roundings to 16 bits: the scores (as any attention's weights), Z as an
// operand, and the output; W is split into two bfloat16 terms (16 bits of the
// product of a value and a power), or three (24 bits) where states are an
// output, so that 32-bit states keep 32-bit accuracy.
//
// A block walks one segment of one head: the copy engine fills a ring of row
// tiles and empties the outputs', one thread issues the products, and warps
// take the steps between them -- state and W (8 warps), scores (2), output (4)
// -- each at its own chunk, through barriers in shared memory.  Two heads of up
// to 64 keys and values share a block, a head in each half of the lanes.
//
// Measured: 65537 rows of 16 heads of 128 in 300 us: the segments' states in 106
// (k and v, 0.54 GB at 5.1 TB/s), their joining in 16, the outputs in 185 (1.07
// GB at 5.8 TB/s, 86% of copy bandwidth), so the second reading of k and v is
// what it costs to walk one long grid on all multiprocessors.  32 grids of 2048
// rows, 16 heads of 64, walked whole: 110 us, 4.9 TB/s.  With few grids the
// longest one's chain bounds it, about 2700 clocks a chunk of two heads, in
// which the tensor pipe is busy half of the time and the warps of the state,
// which make W too, without a pause: 124807 rows in 14 unequal grids, 8 heads of
// 64, 162 us, the three sums of the gradient 282 us.
#include <cstring>

#include "tb_linattn.cuh"
#include "tb_linattn_scan.cuh"
#include "tb_seq.cuh"
#include "tb_linattn_tc.cuh"

namespace tb {
namespace {

constexpr int kOutTile = 4096;    // 64 rows x 64 bytes
// A ring of stages of two tiles each of B, C and A (which states do without):
// what the copies are ahead by has to cover a chunk's time in the block and the
// memory's latency (three stages stalled the segment states every third chunk:
// 124 us for the states of a 65537-token prompt, 106 with six).
constexpr int kMaxStages = 6;
constexpr int stages_of(bool states) { return states ? 6 : 3; }
constexpr int stage_bytes(bool states) { return (states ? 4 : 6) * kTile; }
// Warps: 8 of the state, the copies, the products, 2 of the scores (lanes 64 to
// 127), 4 of the output, and for pairs of heads 2 more of the scores.  Sixteen
// leave 128 registers a thread, which the state of 128 keys and the blocks of W
// need; pairs hold half as many keys.  Where only states are made, 8 other warps
// make W: together they took one warp's turn a chunk each (2400 clocks).
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpScores = 10, kWarpOut = 12, kWarpScores2 = 16;
constexpr int threads_of(bool pair, bool states) { return (states || pair ? 18 : 16) * 32; }

// Blocks in which a wait gave up (a bug, or a GPU that stands still) since the
// library was loaded: read by linear_gave_up and never cleared, so that no
// reader takes another one's report.
__device__ unsigned int g_gave_up;

enum Bars {
  kFull = 0, kEmpty = kFull + kMaxStages, kSReady = kEmpty + kMaxStages, kSFull, kWFull, kWFree = kWFull + 2,
  kKvReady = kWFree + 2, kKvFree = kKvReady + 2, kStFull = kKvFree + 2, kStFree, kOReady, kOFree = kOReady + 2, kZeros = kOFree + 2, kDrain, kBars
};

struct Shared {
  uint64_t bar[kBars];
  uint32_t tmem;
  volatile uint32_t gave_up;
  volatile uint32_t bad[kMaxStages];  // chunk + 1 whose values are not all finite
  LinSegment seg;
  // powers for the rows of a chunk, 0 past the 64th; per head, copy s starts at row s
  __align__(8) float w[2][2][2 * kC + 2];  // fold decay^(31-m), reverse: fold decay^(m-32)
  __align__(8) float o[2][2][2 * kC + 2];  // mul decay^(m-31), reverse: mul decay^(32-m)
  uint2 w2[2][2][kC + 1];                  // rows 2 m, 2 m + 1 of w as bfloat16 pairs: the value, and what it leaves
};

// Adds the scores times c_j of the rows j whose value is not finite to the
// rows i that see them, in a warp's staged output of 32 values (the product
// had zeros in their place).  sign: of the problem's scale.
__device__ __noinline__ void add_not_finite(uint32_t stage, uint32_t scores, uint32_t c_tile, int n, bool reverse,
                                            float sign) {
  const int lane = threadIdx.x & 31, v = ((threadIdx.x >> 5) & 1) * 32 + lane;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const float c = shared_bf16(tile_at(c_tile, j, v));
    if (!not_finite(c)) continue;
#pragma unroll 1
    for (int i = reverse ? 0 : j; i <= (reverse ? j : n - 1); ++i) {
      const uint32_t at = stage + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2;
      const float o = fmaf(shared_bf16(tile_at(scores, i, j)) * sign, c, shared_bf16(at));
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)(bf16x2(o, o) & 0xffffu)) : "memory");
    }
  }
}

// The same for the state: adds b_j c_j of those rows to (B^T W)^T in tensor
// memory, the weights of a value that is not finite left out.  The columns
// hold keys from `key` on; the lane's value is v % 64 of the tile.
__device__ __noinline__ void add_not_finite_state(uint32_t columns, int keys, uint32_t b_tile, int key, uint32_t c_tile,
                                                  int n, float sign) {
  const int v = ((threadIdx.x >> 5) & 1) * 32 + (threadIdx.x & 31);
#pragma unroll 1
  for (int k0 = 0; k0 < keys; k0 += 16) {
    uint32_t y[16];
    tmem_ld16(columns + k0, y);
    tmem_wait_ld();
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const float c = shared_bf16(tile_at(c_tile, j, v));
      if (!not_finite(c)) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int k = key + k0 + i;
        y[i] = __float_as_uint(
            fmaf(shared_bf16(tile_at(b_tile + (k >> 6) * kTile, j, k & 63)) * sign, c, __uint_as_float(y[i])));
      }
    }
    __syncwarp();
    tmem_st16(columns + k0, y);
  }
  tmem_wait_st();
}

// The recurrence by the block's first 8 warps; apart, so that its registers are
// not the chunks'.
template <int KS>
__device__ __noinline__ void walk_rows(const LinLaunch& l, const LinProblem& p, const LinSegment& seg, int h,
                                       float* s_rows) {
  scan_walk<__nv_bfloat16, KS>(l, p, seg, h, s_rows, 256);
}

// kPair: two heads of up to 64 keys and values, one in each half of the 128
// lanes.  Every product then takes both heads' tiles, which lie next to each
// other, as 128 columns: a lane's own head is one half of its columns, the
// other half is not read.  Else one head, of up to 128 (fewer keys and values
// are padded with zeros by the copies).
// kStates: the states of segments alone, without outputs.
template <bool kPair, int kTerms, bool kStates>
__global__ void __launch_bounds__(threads_of(kPair, kStates), 1) k_chunks(const __grid_constant__ ChunkLaunch g) {
  constexpr int kHeads = kPair ? 2 : 1, kStages = stages_of(kStates), kStageBytes = stage_bytes(kStates);
  constexpr int kTileB = 0, kTileC = 2, kTileA = 4;        // of a stage
  constexpr int kKeys = kPair ? 64 : 128;                  // of a head
  constexpr int kRows = kHeads * kC;                       // columns of the products over rows
  // Buffers in tensor memory: of W^T, of its product with B, of the output.
  constexpr int kWs = kStates || (!kPair && kTerms == 2) ? 2 : 1, kKvs = kStates ? 2 : 1, kOs = kPair ? 1 : 2;
  constexpr uint32_t kColS = 0, kColO = kRows, kColKv = kStates ? 0 : kColO + kOs * kRows, kColW = kColKv + 128 * kKvs,
                     kColZ = kColW + 32 * kTerms * kWs;
  static_assert(kColZ + kKeys / 2 <= 512, "tensor memory");

  if (kStates) let_next_kernel_start();
  extern __shared__ char s_raw[];
  __shared__ Shared s;
  // two score tiles for each head, then the stages (with one head the product A B^T reads the 8 KB before A too, C),
  // then the outputs
  const uint32_t tiles = (smem_addr(s_raw) + 1023) & ~1023u;
  const uint32_t stage0 = tiles + (kStates ? 0 : 2 * kHeads * kTile);

  const LinLaunch& l = g.l;
  // blocks in the order of their segments, longest grids first where they are walked whole
  const int walks = (l.heads + kHeads - 1) / kHeads;
  const int slot0 = blockIdx.x / (walks * l.n), walk = blockIdx.x % (walks * l.n), problem = walk / walks;
  const LinProblem& p = l.p[problem];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int h0 = (walk - problem * walks) * kHeads;
  auto bar = [&](int i) { return smem_addr(&s.bar[i]); };
  const bool reverse = p.reverse;
  // The heads that go by chunks, and their decays; the recurrence takes the others that exist.
  float decay[kHeads];
  bool present[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const float d = h0 + i < l.heads ? l.decay[h0 + i] : 0.f;
    present[i] = d >= kSteep && d <= 1.f / kSteep;
    decay[i] = present[i] ? d : 1.f;
  }

  if (warp == 0) {
    const LinSegment seg = lin_segment(l, l.sorted ? lin_grid_of_rank(l, slot0) : slot0);
    if (lane == 0) s.seg = seg;
  } else if (warp == 1) {
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        mbar_init(bar(kFull + i), 1);
        mbar_init(bar(kEmpty + i), kStates ? 17 : 13);  // products, state warps, W's or output warps
        s.bad[i] = 0;
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(kWFull + i), 8);
        mbar_init(bar(kWFree + i), 1);
        mbar_init(bar(kKvReady + i), 1);
        mbar_init(bar(kKvFree + i), 8);
        mbar_init(bar(kOReady + i), 1);
        mbar_init(bar(kOFree + i), 4);
      }
      mbar_init(bar(kSReady), 1);
      mbar_init(bar(kSFull), kPair ? 4 : 2);
      mbar_init(bar(kStFull), 8);
      mbar_init(bar(kStFree), 1);
      mbar_init(bar(kZeros), 8);
      mbar_init(bar(kDrain), 1);
      s.gave_up = 0;
      fence_mbar_init();
    }
  } else if (warp == kWarpMma) {
    tmem_alloc(smem_addr(&s.tmem), 512);
  } else if (warp >= 4 && warp < 8) {
#pragma unroll
    for (int hd = 0; hd < kHeads; ++hd) {
      const float log = log2f(decay[hd]);
#pragma unroll 1
      for (int j = threadIdx.x - 128; j < 2 * (2 * kC + 2); j += 128) {
        const int c = j & 1, i = j >> 1, m = i + c;
        const float x = reverse ? (float)(m - 32) : (float)(31 - m);
        const float w0 = m < kC ? p.fold * exp2f(x * log) : 0.f;
        s.w[hd][c][i] = w0;
        s.o[hd][c][i] = m < kC ? p.mul * exp2f(-x * log) : 0.f;
        if ((i & 1) == 0) {
          const float w1 = m + 1 < kC ? p.fold * exp2f((reverse ? x + 1.f : x - 1.f) * log) : 0.f;
          const uint32_t hi = bf16x2(w0, w1);
          s.w2[hd][c][i / 2] = make_uint2(hi, bf16x2(w0 - low(hi), w1 - high(hi)));
        }
      }
    }
  } else if (!kStates && warp >= kWarpScores) {
    constexpr int first = kWarpScores * 32;
    lin_zero_share<uint16_t>(l, p, slot0, h0, min(kHeads, l.heads - h0), threadIdx.x - first, threads_of(kPair, kStates) - first);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const LinSegment seg = s.seg;
  const uint32_t tmem = s.tmem;
  // a slot without a segment, or a segment whose state nobody reads
  const bool idle = seg.grid < 0 || (kStates && seg.index + 1 == seg.count && !p.last);
  const bool any = present[0] || present[kHeads - 1];
  const int chunks = idle || !any ? 0 : (seg.len + kC - 1) / kC;
  auto rows_of = [&](int t) { return min(kC, seg.len - t * kC); };
  auto row_of = [&](int t) {
    return reverse ? seg.end - seg.first - (int64_t)t * kC - rows_of(t) : seg.begin + seg.first + (int64_t)t * kC;
  };
  auto wait = [&](int i, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar(i), parity & 1, &s.gave_up));
  };
  auto arrive = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(i));
  };
  const int value_tiles = kPair || p.V > 64 ? 2 : 1;
  // A quarter of the lanes: its head, its first value there, whether it has any.
  const int quarter = warp & 3, head = kPair ? quarter >> 1 : 0, value0 = (kPair ? quarter & 1 : quarter) * 32;
  const bool live = (kPair && head ? present[kHeads - 1] : present[0]) && value0 < p.V;
  const uint32_t lanes = tmem + ((uint32_t)quarter << 21);
  const int h = h0 + head;

  const int half = kStates && warp >= kWarpScores ? (warp - kWarpScores) >> 2 : warp >> 2;  // of the keys, of a chunk's rows
  // W^T of chunk x: its terms in registers, then in tensor memory.
  uint32_t y[2][kTerms][8];
  auto make_w = [&](int x) {
    const int st = x % kStages, n = rows_of(x);
    const uint32_t at = stage0 + st * kStageBytes;
    if (!wait(kFull + st, x / kStages)) return false;
    if (n < kC) {
      // rows past the segment belong to others: no NaN of theirs may meet the zeros that stand for them
#pragma unroll 1
      for (int i = threadIdx.x - (kStates ? kWarpScores * 32 : 0); i < (2 + value_tiles) * (kC - n) * 8; i += 256) {
        const int blk = i / ((kC - n) * 8), r = i % ((kC - n) * 8);
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                         at + blk * kTile + n * 128 + r * 16),
                     "r"(0)
                     : "memory");
      }
      fence_async_smem();
      arrive(kZeros);  // once: only the last chunk is short
      if (!wait(kZeros, 0)) return false;
    }
    if (live) {
      // this warp's 32 values x its half of the rows, as 8 x 8 blocks read across: a register is two rows of a
      // value
      const int skip = reverse ? kC - n : 0;
      const float* w = s.w[head][skip & 1] + (skip & ~1) + half * 32 + 2 * (lane & 3);
      const uint2* w2 = s.w2[head][skip & 1] + skip / 2 + half * 16 + (lane & 3);
      const int r = half * 32 + (lane >> 4) * 8 + (lane & 7);
      const uint32_t rows = at + (kTileC + (quarter >> 1)) * kTile + r * 128;
#pragma unroll
      for (int g16 = 0; g16 < 2; ++g16) {
        uint32_t c[8];
        const uint32_t from = rows + ((((quarter & 1) * 4 + g16 * 2 + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
        ldmatrix_trans4(from, c[0], c[1], c[2], c[3]);
        ldmatrix_trans4(from + 16 * 128, c[4], c[5], c[6], c[7]);
        uint32_t finite = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) finite = fma_bf16x2(c[i], 0u, finite);
        if (__any_sync(0xffffffffu, not_finite(low(finite)) || not_finite(high(finite)))) {
          // 0 x infinity of a later row is no part of an earlier row's sum: the products take zeros, and the
          // warps of the output and of the state add these values to what sees them
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (not_finite(low(c[i]))) c[i] &= 0xffff0000u;
            if (not_finite(high(c[i]))) c[i] &= 0xffffu;
          }
          s.bad[st] = x + 1;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (kTerms == 2) {
            // c (w + w') = hi + lo: hi = round(c w), c w - hi is exact in 16 bits
            const uint2 wv = w2[(i / 2) * 4];
            y[g16][0][i] = mul_bf16x2(c[i], wv.x);
            y[g16][1][i] = fma_bf16x2(c[i], wv.y, fma_bf16x2(c[i], wv.x, y[g16][0][i] ^ 0x80008000u));
          } else {
            const float2 wv = *reinterpret_cast<const float2*>(w + (i / 2) * 8);
            f32x2 e = mul2(pair(low(c[i]), high(c[i])), pair(wv.x, wv.y));
#pragma unroll
            for (int term = 0; term < kTerms; ++term) {
              const uint32_t x2 = bf16x2(halves(e).x, halves(e).y);
              y[g16][term][i] = x2;
              if (term + 1 < kTerms) e = fma2(pair(low(x2), high(x2)), pair(-1.f, -1.f), e);
            }
          }
        }
      }
    }
    return true;
  };
  auto put_w = [&](int x) {
    if (x >= kWs && !wait(kWFree + x % kWs, x / kWs - 1)) return false;
    tc_fence_after();
    if (live) {
#pragma unroll
      for (int g16 = 0; g16 < 2; ++g16) {
        const uint32_t to = lanes + ((uint32_t)g16 << 20) + kColW + x % kWs * 32 * kTerms + half * 16;
#pragma unroll
        for (int term = 0; term < kTerms; ++term) tmem_st_16x16(to + term * 32, y[g16][term]);
      }
      tmem_wait_st();
    }
    tc_fence_before();
    arrive(kWFull + x % kWs);
    return true;
  };

  if (warp == kWarpTma) {
    if (elect_one()) {
      const CUtensorMap* ma = &g.map[g.a[problem]];
      const CUtensorMap* mb = &g.map[g.b[problem]];
      const CUtensorMap* mc = &g.map[g.c[problem]];
      const uint32_t bytes = ((kStates ? 2 : 4) + value_tiles) * kTile;
      int t = 0;
#pragma unroll 1
      for (; t < chunks; ++t) {
        const int st = t % kStages;
        if (t >= kStages && !mbar_wait(bar(kEmpty + st), (t / kStages - 1) & 1, &s.gave_up)) break;
        const uint32_t at = stage0 + st * kStageBytes;
        const int row = (int)row_of(t);
        mbar_expect(bar(kFull + st), bytes);
        auto load = [&](int tile, const CUtensorMap* map, int i) {
          tma_load_3d(at + (tile + i) * kTile, map, kPair ? 0 : 64 * i, kPair ? h0 + i : h0, row, bar(kFull + st));
        };
        for (int i = 0; i < value_tiles; ++i) load(kTileC, mc, i);
        for (int i = 0; i < 2; ++i) load(kTileB, mb, i);
        if (!kStates)
          for (int i = 0; i < 2; ++i) load(kTileA, ma, i);
      }
      if (s.gave_up) {  // copies in flight land before the block ends
        for (int i = t > kStages ? t - kStages : 0; i < t; ++i) {
          uint32_t flag = 0;
          mbar_wait(bar(kFull + i % kStages), (i / kStages) & 1, &flag);
        }
      }
    }
  } else if (warp == kWarpMma) {
    if (chunks && elect_one()) {
      constexpr uint32_t kRowDesc = mma_desc(128, kRows, false);
      constexpr uint32_t kKvDesc = mma_desc(128, 128, true);
      auto one = [&](int i, uint32_t parity) { return mbar_wait(bar(i), parity & 1, &s.gave_up); };
      // A B^T: the rows of one head in lanes 64 to 127 (lanes 0 to 63 get whatever lies before A), of two heads in
      // 0 to 63 and 64 to 127
      auto scores = [&](int t) {
        const uint32_t at = stage0 + t % kStages * kStageBytes;
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k) {
          const uint32_t off = (k >> 2) * kTile + (k & 3) * 32;
          mma_ss(tmem + kColS, smem_desc(at + (kPair ? kTileA : kTileA - 1) * kTile + off, 16),
                 smem_desc(at + kTileB * kTile + off, 16), kRowDesc, k > 0);
        }
        mma_commit(bar(kSReady));
      };
      bool ok = one(kFull, 0);
      if (ok && rows_of(0) < kC) ok = one(kZeros, 0);
      tc_fence_after();
      if (ok && !kStates) scores(0);
#pragma unroll 1
      for (int t = 0; ok && t < chunks; ++t) {
        const int st = t % kStages, wb = t % kWs, kv = t % kKvs;
        const uint32_t at = stage0 + st * kStageBytes;
        const int ob = t % kOs;
        const uint32_t w = tmem + kColW + wb * 32 * kTerms, o = tmem + kColO + ob * kRows;
        // W^T B (W full: the tile is)
        ok = one(kWFull + wb, t / kWs) && (t < kKvs || one(kKvFree + kv, t / kKvs - 1));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int term = 0; term < kTerms; ++term)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_ts(tmem + kColKv + kv * 128, w + term * 32 + j * 8, smem_desc(at + kTileB * kTile + j * 2048, kTile), kKvDesc,
                   term > 0 || j > 0);
        mma_commit(bar(kKvReady + kv));
        if (!kStates) {
          // Z^T A^T
          ok = one(kStFull, t) && (t < kOs || one(kOFree + ob, t / kOs - 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ts(o, tmem + kColZ + k * 8, smem_desc(at + kTileA * kTile + (k >> 2) * kTile + (k & 3) * 32, 16), kRowDesc, k > 0);
          mma_commit(bar(kStFree));
          // the next chunk's scores, once this chunk's are out of tensor memory
          ok = one(kSFull, t) && (t + 1 >= chunks || one(kFull + (t + 1) % kStages, (t + 1) / kStages));
          if (ok && t + 1 < chunks && rows_of(t + 1) < kC) ok = one(kZeros, 0);
          if (!ok) break;
          tc_fence_after();
          if (kWs == 2 && t + 1 < chunks) scores(t + 1);
          // W^T scores^T (two terms of W are more than the scores have)
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_ts(o, w + term * 32 + j * 8, smem_desc(tiles + (t & 1) * kHeads * kTile + j * 32, 16), kRowDesc, true);
          mma_commit(bar(kOReady + ob));
        }
        mma_commit(bar(kWFree + wb));
        if (kWs == 1 && !kStates && t + 1 < chunks) scores(t + 1);  // after what frees W^T
        mma_commit(bar(kEmpty + st));
      }
      if (!ok) {  // products in flight finish before tensor memory is given back
        uint32_t flag = 0;
        mma_commit(bar(kDrain));
        mbar_wait(bar(kDrain), 0, &flag);
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ state, W
    constexpr int NK = kKeys / 2;  // keys of a thread
    const int v = value0 + lane;
    const int64_t state_at = ((int64_t)seg.grid * l.heads + h) * p.K * p.V;
    float* seg_state = p.seg ? p.seg + ((int64_t)seg.slot * l.heads + h) * p.K * p.V : nullptr;
    const float log = log2f(kPair && head ? decay[kHeads - 1] : decay[0]);
    const float enter = chunks ? exp2f((reverse ? 31.f : 32.f) * log) : 1.f, full = exp2f(64.f * log);
    if (l.phase == 2) wait_for_last_kernel();  // the states that enter
    f32x2 u[NK / 2];  // Z, by pairs of keys
    {
      const float* from = l.phase == 2 ? seg_state : p.first ? p.first + state_at : nullptr;
      const int64_t step = l.phase == 2 ? p.V : p.first_k;
      const int keys = kStates || idle || !live || !from || v >= p.V ? 0 : p.K - half * NK;
      if (from) from += half * NK * step + v * (l.phase == 2 ? 1 : p.first_v);
#pragma unroll
      for (int i = 0; i < NK; i += 2, from += 2 * step)
        u[i / 2] = pair(i < keys ? from[0] * enter : 0.f, i + 1 < keys ? from[step] * enter : 0.f);
    }
    // The state after chunk t.
    auto update = [&](int t) {
      const int st = t % kStages, n = rows_of(t);
      if (!wait(kKvReady + t % kKvs, t / kKvs)) return false;
      tc_fence_after();
      // after the last chunk the state itself: decay^n X + decay^(n-e-r) B^T W
      const float d = t + 1 < chunks ? full : exp2f((float)(n - (reverse ? 31 : 32)) * log);
      if (live) {
        if (s.bad[st] == (uint32_t)t + 1) {
          const uint32_t at = stage0 + st * kStageBytes;
          add_not_finite_state(lanes + kColKv + t % kKvs * 128 + head * 64 + half * NK, NK, at + (kTileB + head) * kTile,
                               half * NK, at + (kTileC + (quarter >> 1)) * kTile, n, sign_of(p.fold));
        }
        const f32x2 d2 = pair(d, d);
#pragma unroll
        for (int k0 = 0; k0 < NK; k0 += 16) {
          uint32_t z[16];
          tmem_ld16(lanes + kColKv + t % kKvs * 128 + head * 64 + half * NK + k0, z);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; i += 2)
            u[(k0 + i) / 2] = mul2(add2(u[(k0 + i) / 2], pair(__uint_as_float(z[i]), __uint_as_float(z[i + 1]))), d2);
        }
      }
      tc_fence_before();
      arrive(kKvFree + t % kKvs);
      arrive(kEmpty + st);
      return true;
    };
    // Z^T as chunk x's operand.
    auto put_z = [&](int x) {
      if (x > 0 && !wait(kStFree, x - 1)) return false;
      tc_fence_after();
      if (live) {
#pragma unroll
        for (int k0 = 0; k0 < NK; k0 += 32) {
          uint32_t z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = bf16x2(halves(u[k0 / 2 + i]).x, halves(u[k0 / 2 + i]).y);
          tmem_st16(lanes + kColZ + (half * NK + k0) / 2, z);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      arrive(kStFull);
      return true;
    };
    // With one buffer of W^T it is free only after the chunk's last product: the state's turn comes before, and a
    // pair's state leaves the registers to hold W^T meanwhile.
    constexpr bool kAhead = kWs == 2 || kPair;
#pragma unroll 1
    for (int t = -1; t < chunks; ++t) {
      const bool more = t + 1 < chunks;
      if (kAhead && !kStates && more && !make_w(t + 1)) break;
      if (kWs == 2 && !kStates && more && !put_w(t + 1)) break;
      if (t >= 0 && !update(t)) break;
      if (!kStates && more && !put_z(t + 1)) break;
      if (!kAhead && more && !make_w(t + 1)) break;
      if (kWs == 1 && more && !put_w(t + 1)) break;
    }
    float* dst = kStates ? seg_state : l.phase == 0 && p.last ? p.last + state_at : nullptr;
    if (!idle && live && dst && !s.gave_up && v < p.V) {
      dst += half * NK * p.V + v;
#pragma unroll
      for (int i = 0; i < NK; i += 2, dst += 2 * p.V) {
        if (i < p.K - half * NK) dst[0] = halves(u[i / 2]).x;
        if (i + 1 < p.K - half * NK) dst[p.V] = halves(u[i / 2]).y;
      }
    }
  } else if (kStates) {
    // ------------------------------------------------------------------- W
#pragma unroll 1
    for (int x = 0; x < chunks; ++x) {
      if (!make_w(x) || !put_w(x)) break;
      arrive(kEmpty + x % kStages);
    }
  } else if (warp < kWarpOut || warp >= kWarpScores2) {
    // -------------------------------------------------------------- scores
    // Rows past a segment's end need no mask: their b are zeros before the scores are computed, and rows i past it
    // are not written.
    const int block = warp & 1, i = block * 32 + lane;
    uint32_t diagonal[16];  // of pairs of columns in the 32 x 32 block on the diagonal
#pragma unroll
    for (int j = 0; j < 16; ++j)
      diagonal[j] = ((reverse ? 2 * j >= lane : 2 * j <= lane) ? 0xffffu : 0u) |
                    ((reverse ? 2 * j + 1 >= lane : 2 * j + 1 <= lane) ? 0xffff0000u : 0u);
#pragma unroll 1
    for (int t = 0; t < chunks; ++t) {
      if (!wait(kSReady, t)) break;
      // the output warps may still read the tile's last scores where they add values that are not finite
      if (t >= 2 && s.bad[(t - 2) % kStages] == (uint32_t)t - 1 && !wait(kOFree + t % kOs, t / kOs - 1)) break;
      tc_fence_after();
      const uint32_t row = tiles + ((t & 1) * kHeads + head) * kTile + i * 128;
#pragma unroll
      for (int b = 0; b < 2; ++b) {  // columns 32 b to 32 b + 31
        const bool some = reverse ? b >= block : b <= block;
        if (!some && t >= 2) continue;  // the tile's other half stays zero
        uint32_t x[32], y[16];
        if (some) {
          tmem_ld32(lanes + kColS + head * 64 + 32 * b, x);
          tmem_wait_ld();
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          y[j] = bf16x2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
          y[j] = !some ? 0u : b == block ? y[j] & diagonal[j] : y[j];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + (((b * 4 + q) ^ (i & 7)) << 4)),
                       "r"(y[4 * q]), "r"(y[4 * q + 1]), "r"(y[4 * q + 2]), "r"(y[4 * q + 3])
                       : "memory");
      }
      fence_async_smem();
      tc_fence_before();
      arrive(kSFull);
    }
  } else {
    // -------------------------------------------------------------- output
    const uint32_t out0 = stage0 + kStages * kStageBytes + quarter * 2 * kOutTile;
    const CUtensorMap* map = &g.map[kLinMaxRows + problem];
#pragma unroll 1
    for (int t = 0; t < chunks; ++t) {
      const int st = t % kStages, n = rows_of(t);
      if (!wait(kOReady + t % kOs, t / kOs)) break;
      tc_fence_after();
      if (live) {
        const int skip = reverse ? kC - n : 0;
        const float* w = s.o[head][skip & 1] + (skip & ~1) + 2 * (lane & 3);
        const bool bad = s.bad[st] == (uint32_t)t + 1;
        const uint32_t buf = out0 + (t & 1) * kOutTile;
        const int row = (lane >> 4) * 8 + (lane & 7);
        if (lane == 0) tma_store_wait<1>();
        __syncwarp();
        uint32_t x[2][32];
        const uint32_t from = lanes + kColO + t % kOs * kRows + head * 64;
        tmem_ld_16x64(from, x[0]);
        tmem_ld_16x64(from + (1u << 20), x[1]);
        tmem_wait_ld();
        if (!bad) {
          tc_fence_before();
          arrive(kOFree + t % kOs);
        }
#pragma unroll
        for (int m = 0; m < 8; m += 2) {
          const float2 w0 = *reinterpret_cast<const float2*>(w + 8 * m), w1 = *reinterpret_cast<const float2*>(w + 8 * m + 8);
          const f32x2 w0p = pair(w0.x, w0.y), w1p = pair(w1.x, w1.y);
#pragma unroll
          for (int g16 = 0; g16 < 2; ++g16) {
            const uint32_t* y = x[g16] + 4 * m;
            auto both = [&](int i, f32x2 wp) {
              const float2 o = halves(mul2(pair(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), wp));
              return bf16x2(o.x, o.y);
            };
            stmatrix_trans4(buf + row * 64 + (((g16 * 2 + ((lane >> 3) & 1)) ^ ((row >> 1) & 3)) << 4) + m * 8 * 64,
                            both(0, w0p), both(2, w0p), both(4, w1p), both(6, w1p));
          }
        }
        __syncwarp();
        if (bad) {
          add_not_finite(buf, tiles + ((t & 1) * kHeads + head) * kTile,
                         stage0 + st * kStageBytes + (kTileC + (quarter >> 1)) * kTile, n, reverse, sign_of(p.mul) * sign_of(p.fold));
          tc_fence_before();
          arrive(kOFree + t % kOs);
        }
        const int64_t row0 = row_of(t);
        if (n == kC) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) tma_store_3d(map, value0, h, (int)row0, buf);
        } else {
          // the rows that follow are not this segment's: plain stores
#pragma unroll 1
          for (int i = lane; i < n * 4; i += 32) {
            const int rr = i >> 2, v = value0 + (i & 3) * 8;
            uint4 o;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                         : "r"(buf + rr * 64 + (((i & 3) ^ ((rr >> 1) & 3)) << 4)));
            if (v < p.V) *reinterpret_cast<uint4*>((__nv_bfloat16*)p.out + (row0 + rr) * p.o_row + h * p.o_head + v) = o;
          }
        }
      } else {
        tc_fence_before();
        arrive(kOFree + t % kOs);
      }
      arrive(kEmpty + st);
    }
    if (lane == 0) tma_store_wait<0>();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && s.gave_up) atomicAdd(&g_gave_up, 1u);
  if (warp == kWarpMma) tmem_free(tmem, 512);
  if (idle || warp >= 8) return;
  if (l.phase == 2) wait_for_last_kernel();
#pragma unroll 1
  for (int i = 0; i < kHeads; ++i)
    if (!(i ? present[kHeads - 1] : present[0]) && h0 + i < l.heads)
      walk_rows<kKeys / 4>(l, p, s.seg, h0 + i, reinterpret_cast<float*>(s_raw + (tiles - smem_addr(s_raw))));
}

template <bool kPair, int kTerms, bool kStates>
cudaError_t go(const ChunkLaunch& g, cudaStream_t s) {
  constexpr int bytes = 1024 + stages_of(kStates) * stage_bytes(kStates) +
                        (kStates ? 0 : (kPair ? 4 : 2) * kTile + 4 * 2 * kOutTile);
  static_assert(bytes > 116 * 1024 && bytes < 222 * 1024, "one block a multiprocessor: tensor memory is not shared");
  static std::atomic<bool> ready[kMaxDevices];
  const cudaError_t e = allow_shared(k_chunks<kPair, kTerms, kStates>, bytes, ready);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (int64_t)g.l.segments * (kPair ? (g.l.heads + 1) / 2 : g.l.heads) * g.l.n;
  return launch_early(k_chunks<kPair, kTerms, kStates>, (unsigned)blocks, threads_of(kPair, kStates), bytes, s,
                      g.l.phase == 2, g);
}

typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                           const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                           CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return (Encode)f;
  }();
  return fn;
}

// Rows [tokens, heads, size] as the copy engine takes them, a box of 64 rows of
// one head: 64 elements of it read, or 32 written.  False where it cannot.
bool row_map(CUtensorMap* m, const void* at, int size, int heads, int64_t tokens, int64_t row, int64_t head, int box_size) {
  if (!encoder() || ((uintptr_t)at & 15)) return false;
  // a stride that nothing is reached by still has to be one the encoding takes
  if (heads == 1) head = size;
  if (tokens == 1) row = (int64_t)heads * size;
  if (head <= 0 || row <= 0 || head % 8 || row % 8 || head >= 1ll << 38 || row >= 1ll << 38) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)size, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)row * 2};
  const cuuint32_t box[3] = {(cuuint32_t)box_size, 1, kC}, step[3] = {1, 1, 1};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(at), dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, box_size == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

__global__ void __launch_bounds__(32) k_wait_selftest(uint32_t polls) {
  __shared__ uint64_t bar;
  __shared__ volatile uint32_t gave_up;
  if (mbar_selftest(&bar, &gave_up, polls) && threadIdx.x == 0) atomicAdd(&g_gave_up, 1u);
}

}  // namespace

bool linear_chunk_plan(ChunkLaunch& g) {
  const LinLaunch& l = g.l;
  struct Rows {
    const void* at;
    int size;
    int64_t row, head;
  } known[kLinMaxRows];
  int n = 0;
  auto find = [&](const Rows& x, uint8_t* to) {
    for (int i = 0; i < n; ++i)
      if (known[i].at == x.at && known[i].size == x.size && known[i].row == x.row && known[i].head == x.head) {
        *to = (uint8_t)i;
        return true;
      }
    if (n == kLinMaxRows || !row_map(&g.map[n], x.at, x.size, l.heads, l.tokens, x.row, x.head, 64)) return false;
    known[n] = x;
    *to = (uint8_t)n++;
    return true;
  };
  if (l.type != TB_TYPE_BF16) return false;
  for (int i = 0; i < l.n; ++i) {
    const LinProblem& p = l.p[i];
    if (p.K % 8 || p.V % 8 || p.reverse != p.late || (p.reverse ? p.mul : p.fold) != 1.f) return false;
    if (!find({p.a, p.K, p.a_row, p.a_head}, &g.a[i]) || !find({p.b, p.K, p.b_row, p.b_head}, &g.b[i]) ||
        !find({p.c, p.V, p.c_row, p.c_head}, &g.c[i]) ||
        !row_map(&g.map[kLinMaxRows + i], p.out, p.V, l.heads, l.tokens, p.o_row, p.o_head, 32))
      return false;
  }
  return true;
}

cudaError_t launch_linear_chunks(const void* args, cudaStream_t s) {
  const ChunkLaunch& g = *(const ChunkLaunch*)args;
  const bool pair = linear_pairs(g.l.p[0].K, g.l.p[0].V);
  bool exact = false;
  for (int i = 0; i < g.l.n; ++i) exact = exact || g.l.p[i].last;
  if (g.l.phase == 1) {
    if (pair) return exact ? go<true, 3, true>(g, s) : go<true, 2, true>(g, s);
    return exact ? go<false, 3, true>(g, s) : go<false, 2, true>(g, s);
  }
  if (g.l.phase == 2) exact = false;  // the states that leave come from phase 1
  if (pair) return exact ? go<true, 3, false>(g, s) : go<true, 2, false>(g, s);
  return exact ? go<false, 3, false>(g, s) : go<false, 2, false>(g, s);
}

cudaError_t linear_selftest(const void* args, cudaStream_t s) {
  k_wait_selftest<<<1, 32, 0, s>>>(*(const uint32_t*)args);
  return cudaGetLastError();
}

cudaError_t linear_gave_up(cudaStream_t s, unsigned int* count) {
  void* at = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&at, g_gave_up);
  if (e == cudaSuccess) e = cudaMemcpyAsync(count, at, sizeof *count, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e;
}

}  // namespace tb
