// C entry points of the sequence operators: checks of the arguments, the
// choice of a kernel's shape, the launches.  No allocation and no wait.
#include <atomic>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>

#include "tb_seq.h"

using namespace tb;

namespace {

constexpr int64_t kMaxRows = (1ll << 31) - 1;

#define TB_SEQ_CUDA(expr)                                                                          \
  do {                                                                                             \
    const cudaError_t e_ = (expr);                                                                 \
    if (e_ != cudaSuccess) return seq_fail(TB_ERR_CUDA, "%s: %s", #expr, cudaGetErrorString(e_)); \
  } while (0)

int type_size(int32_t type) { return type == TB_TYPE_F32 ? 4 : 2; }
bool type_ok(int32_t type) { return type >= TB_TYPE_F32 && type <= TB_TYPE_BF16; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
bool whole(int64_t stride, int size) { return stride * size % 16 == 0; }
int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads of a row, groups of elements (vectors, or single elements) of a
// thread and rows of a block of the norm kernels, which exist for `counts`
// groups a thread.  One group while that takes at most `wide` threads; else
// the fewest that take at most `most`, as joining many warps costs a wide row
// more than it loads (60000 rows of 1536 in 16 bits: 6 warps a row 107 us, 3
// warps 83; of 4096: 16 warps 154, 4 warps 150).  Rows of half a warp and less
// share one (67722 rows of 64: 11 us, 17 with a warp each; the gradient 17 and
// 29).  Few rows: one group, for the shortest chain of loads.
struct NormShape {
  int per_row, nv, rows;
};
NormShape norm_shape(bool many, int groups, const int* counts, int n, int wide, int most) {
  NormShape r{};
  for (int i = 0; i < n; ++i) {
    r.nv = counts[i];
    r.per_row = (int)(up(up(groups, counts[i]), 32) * 32);
    while (many && r.per_row <= 32 && r.per_row > 4 && r.per_row / 2 * counts[i] >= groups) r.per_row /= 2;
    if (r.per_row <= (!many ? 512 : i == 0 ? wide : most)) break;
  }
  r.rows = many && r.per_row < 128 ? 128 / r.per_row : 1;
  return r;
}
constexpr int kVecs[] = {1, 2, 4, 8}, kOnes[] = {4, 8, 32};

// Rows of a group through shared memory and buffers for groups: as many rows
// as make whole vectors where two buffers leave room for two blocks on a
// multiprocessor, fewer rows where they are wide, down to a row and a buffer
// (3598 rows of 5819, the gradient in 16 bits: 79 us by single rows, 530 element
// by element).
struct NormGroups {
  int rows, stages;
};
NormGroups norm_groups(int width, int size, int tensors, int fixed) {
  for (int rows = 16 / size; rows; rows /= 2)
    if (norm_group_bytes(width, size, tensors, rows, 2, fixed) <= kNormGroupBytes / 2) return {rows, 2};
  for (int stages = 2; stages; --stages)
    if (norm_group_bytes(width, size, tensors, 1, stages, fixed) <= kNormGroupBytes) return {1, stages};
  return {0, 0};
}
// Blocks, and their threads: the more, the fewer blocks a multiprocessor holds
// (10000 rows of 8191 in 16 bits, one block: the gradient 488 us with 256
// threads, 322 with 1024; 50000 of 777 in 32 bits, three blocks: 113 with 256
// each, 141 with 512).
int norm_group_blocks(int64_t rows, int width, int size, int tensors, NormGroups g, int fixed, int sms, int* threads) {
  int64_t fit = 208 * 1024 / (int64_t)(norm_group_bytes(width, size, tensors, g.rows, g.stages, fixed) + 1024);
  if (fit > 8) fit = 8;
  *threads = fit > 2 ? 256 : fit > 1 ? 512 : 1024;
  const int64_t groups = up(rows, g.rows);
  return (int)(groups < fit * sms ? groups : fit * sms);
}

}  // namespace

int tb::seq_sms() {
  static std::atomic<int> sms[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  int n = sms[dev].load(std::memory_order_relaxed);
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    sms[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

extern "C" {

// ------------------------------------------------------------------- rotary

tb_status tb_rotary(const tb_rotary_args* args, tb_stream stream) {
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "tb_rotary: args is NULL");
  RotaryLaunch r;
  r.a = *args;
  tb_rotary_args& a = r.a;
  if (!type_ok(a.type)) return seq_fail(TB_ERR_INVALID_ARG, "tb_rotary: unknown type %d", a.type);
  if (a.tokens < 0 || a.q_heads < 0 || a.k_heads < 0)
    return seq_fail(TB_ERR_INVALID_ARG, "tb_rotary: negative size");
  if (a.dim < 1 || a.dim > 256 || a.pairs < 1 || 2 * a.pairs > a.dim)
    return seq_fail(TB_ERR_INVALID_ARG, "tb_rotary: %d pairs of a head of %d elements (at most 256)", a.pairs, a.dim);
  if (a.layout < 0 || a.layout > 1) return seq_fail(TB_ERR_INVALID_ARG, "tb_rotary: unknown layout %d", a.layout);
  if (a.axes < 1 || a.axes > 3) return seq_fail(TB_ERR_INVALID_ARG, "tb_rotary: %d position axes (1 to 3)", a.axes);
  if (a.axes > 1) {
    const int64_t two = (int64_t)a.section[0] + a.section[1];
    if (a.section[0] < 0 || a.section[1] < 0 || two > a.pairs || (a.axes == 2 && two != a.pairs))
      return seq_fail(TB_ERR_INVALID_ARG, "tb_rotary: sections %d, %d of %d pairs", a.section[0], a.section[1], a.pairs);
  }
  if (a.tokens == 0 || a.q_heads + (int64_t)a.k_heads == 0) return TB_OK;
  if (a.tokens > kMaxRows || a.q_heads + (int64_t)a.k_heads > 65535)
    return seq_fail(TB_ERR_TOO_LARGE, "tb_rotary: 2^31 tokens or 65536 heads, or more");
  if (!a.positions || !a.turns || (a.q_heads && (!a.q || !a.q_out)) || (a.k_heads && (!a.k || !a.k_out)))
    return seq_fail(TB_ERR_INVALID_ARG, "tb_rotary: bad pointer");
  const int sms = seq_sms();
  if (!sms) return seq_fail(TB_ERR_CUDA, "tb_rotary: no device");
  // vectors of 16 bytes, of 4 elements of 16 bits, or single elements (51649 tokens of 5 heads of 48 in 16 bits with 12
  // pairs that turn: 19 us by vectors of 4, 49 by elements)
  const int size = type_size(a.type);
  auto fits = [&](int vec) {
    auto ok = [&](const void* p, int64_t row, int64_t head) {
      return (uintptr_t)p % (vec * size) == 0 && row % vec == 0 && head % vec == 0;
    };
    return a.pairs % vec == 0 && (a.dim - 2 * a.pairs) % vec == 0 &&
           (!a.q_heads || (ok(a.q, a.q_row, a.q_head) && ok(a.q_out, a.q_out_row, a.q_out_head))) &&
           (!a.k_heads || (ok(a.k, a.k_row, a.k_head) && ok(a.k_out, a.k_out_row, a.k_out_head)));
  };
  r.vec = fits(16 / size) ? 16 / size : fits(4) ? 4 : 1;
  // A block's threads take 4 rows (token, head) each, unless that leaves
  // multiprocessors idle; the table stays within 16 KB.
  const int units = a.pairs / r.vec + (a.dim - 2 * a.pairs) / r.vec;
  const int heads = a.q_heads + a.k_heads;
  int64_t per = 4ll * (256 / units) / heads;
  const int64_t fit = 16384 / (8 * a.pairs);
  if (per > fit) per = fit;
  if (per > a.tokens / (4 * sms)) per = a.tokens / (4 * sms);
  r.per_block = per < 1 ? 1 : (int)per;
  TB_SEQ_CUDA(seq_launch(kSeqRotary, (cudaStream_t)stream, launch_rotary, &r));
  return TB_OK;
}

// --------------------------------------------------------------------- norm

static tb_status norm_run(const char* what, const tb_norm_args* args, bool layer, const void* bias, tb_stream stream) {
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "%s: args is NULL", what);
  NormLaunch n;
  n.a = *args;
  n.layer = layer;
  n.bias = bias;
  tb_norm_args& a = n.a;
  if (!type_ok(a.type)) return seq_fail(TB_ERR_INVALID_ARG, "%s: unknown type %d", what, a.type);
  if (a.rows < 0 || a.width < 1) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad size", what);
  if (a.width > 16384 || a.rows > kMaxRows)
    return seq_fail(TB_ERR_TOO_LARGE, "%s: rows of %d elements (at most 16384), or 2^31 rows", what, a.width);
  if (a.rows == 0) return TB_OK;
  if (!a.x || !a.weight || !a.y || (a.h_out && !a.residual) || (a.fp8 != 0) != (a.scale != nullptr) || (layer && a.fp8))
    return seq_fail(TB_ERR_INVALID_ARG, "%s: bad pointer", what);
  const int sms = seq_sms();
  if (!sms) return seq_fail(TB_ERR_CUDA, "%s: no device", what);
  const int size = type_size(a.type), vec = 16 / size;
  n.vec = a.width % vec == 0 && aligned16(a.x) && aligned16(a.weight) && aligned16(bias) && whole(a.x_row, size);
  if (a.residual) n.vec = n.vec && aligned16(a.residual) && whole(a.residual_row, size);
  if (a.h_out) n.vec = n.vec && aligned16(a.h_out) && whole(a.h_row, size);
  if (a.fp8) n.vec = n.vec && ((uintptr_t)a.y & (vec - 1)) == 0 && a.y_row % vec == 0;
  else n.vec = n.vec && aligned16(a.y) && whole(a.y_row, size);
  const bool many = a.rows >= 4ll * sms;
  const int tensors = a.residual ? 2 : 1;
  const bool dense = aligned16(a.x) && a.x_row == a.width && a.y_row == a.width && (a.fp8 || aligned16(a.y)) &&
                     (!a.residual || (aligned16(a.residual) && a.residual_row == a.width)) &&
                     (!a.h_out || (aligned16(a.h_out) && a.h_row == a.width));
  const NormGroups groups = !n.vec && (many || a.width > 4096) && dense ? norm_groups(a.width, size, tensors, size) : NormGroups{0, 0};
  n.groups = groups.rows > 0;
  if (n.groups) {
    n.nv = groups.stages;
    n.rows = groups.rows;
    n.blocks = norm_group_blocks(a.rows, a.width, size, tensors, groups, size, sms, &n.per_row);
  } else {
    const NormShape z = n.vec ? norm_shape(many, a.width / vec, kVecs, 4, 128, 128) : norm_shape(many, a.width, kOnes, 3, 32, 128);
    n.per_row = z.per_row, n.nv = z.nv, n.rows = z.rows;
    // blocks stay: as many as run at once, twice that many where a thread has more than a vector
    const int64_t fit = up(z.nv <= 1 ? 1024 : 2048, n.per_row * n.rows), blocks = up(a.rows, n.rows);
    n.blocks = (int)(blocks < sms * fit ? blocks : sms * fit);
  }
  TB_SEQ_CUDA(seq_launch(kSeqNorm, (cudaStream_t)stream, launch_norm, &n));
  return TB_OK;
}

tb_status tb_rms_norm(const tb_norm_args* args, tb_stream stream) {
  return norm_run("tb_rms_norm", args, false, nullptr, stream);
}
tb_status tb_layer_norm(const tb_norm_args* args, const void* bias, tb_stream stream) {
  return norm_run("tb_layer_norm", args, true, bias, stream);
}

// Each block writes a part of dweight, which is read once more.
static int64_t norm_backward_blocks(int64_t rows, int sms) {
  const int64_t most = 6ll * sms;
  return rows < most ? rows : most;
}

int64_t tb_rms_norm_backward_workspace(int64_t rows, int32_t width) {
  if (rows < 0 || width < 1) return 0;
  const int sms = seq_sms();
  return norm_backward_blocks(rows, sms ? sms : 256) * width * (int64_t)sizeof(float);
}

static tb_status norm_backward_run(const char* what, const tb_norm_backward_args* args, bool layer, void* dbias,
                                   tb_stream stream) {
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "%s: args is NULL", what);
  NormBackwardLaunch n;
  n.a = *args;
  n.layer = layer;
  n.dbias = dbias;
  tb_norm_backward_args& a = n.a;
  if (!type_ok(a.type)) return seq_fail(TB_ERR_INVALID_ARG, "%s: unknown type %d", what, a.type);
  if (a.rows < 0 || a.width < 1) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad size", what);
  if (a.width > 16384 || a.rows > kMaxRows)
    return seq_fail(TB_ERR_TOO_LARGE, "%s: rows of %d elements (at most 16384), or 2^31 rows", what, a.width);
  if (!a.dweight || (a.rows && (!a.dy || !a.h || !a.weight || !a.dx || !a.workspace)))
    return seq_fail(TB_ERR_INVALID_ARG, "%s: bad pointer", what);
  const int sms = seq_sms();
  if (!sms) return seq_fail(TB_ERR_CUDA, "%s: no device", what);
  const int64_t most = norm_backward_blocks(a.rows, sms);
  const int64_t need = most * a.width * (int64_t)sizeof(float) * (layer ? 2 : 1);
  if (a.workspace_bytes < need || !aligned16(a.workspace))
    return seq_fail(TB_ERR_INVALID_ARG, "%s: a workspace of %lld bytes, %lld needed", what,
                    (long long)a.workspace_bytes, (long long)need);
  const int size = type_size(a.type), vec = 16 / size;
  n.vec = a.width % vec == 0 && aligned16(a.dy) && aligned16(a.h) && aligned16(a.weight) && aligned16(a.dx) &&
          whole(a.dy_row, size) && whole(a.h_row, size) && whole(a.dx_row, size);
  if (a.dh) n.vec = n.vec && aligned16(a.dh) && whole(a.dh_row, size);
  const bool many = a.rows >= 4ll * sms;
  const int tensors = a.dh ? 3 : 2, fixed = layer ? 12 : 8;
  const bool dense = aligned16(a.dy) && aligned16(a.h) && aligned16(a.dx) && a.dy_row == a.width && a.h_row == a.width &&
                     a.dx_row == a.width && (!a.dh || (aligned16(a.dh) && a.dh_row == a.width));
  const NormGroups groups = !n.vec && (many || a.width > 4096) && dense ? norm_groups(a.width, size, tensors, fixed) : NormGroups{0, 0};
  int64_t blocks;
  n.groups = groups.rows > 0;
  if (n.groups) {
    n.nv = groups.stages;
    n.rows = groups.rows;
    blocks = norm_group_blocks(a.rows, a.width, size, tensors, groups, fixed, sms, &n.per_row);
  } else {
    // dweight takes registers: up to two vectors a thread while the row fits 512
    const NormShape z = n.vec ? norm_shape(many, a.width / vec, kVecs, 4, 256, 512)
                              : norm_shape(many, a.width, kOnes + 1, 2, 128, 128);
    n.per_row = z.per_row, n.nv = z.nv, n.rows = z.rows;
    // a block's parts of dweight meet in shared memory
    while (n.rows > 1 && (int64_t)n.rows * n.per_row * n.nv * (n.vec ? vec : 1) * 4 > 40 * 1024) n.rows /= 2;
    const int64_t fit = sms * up(768, n.per_row * n.rows);
    blocks = up(a.rows, n.rows);
    if (blocks > fit) blocks = fit;
  }
  n.blocks = (int)(blocks < most ? blocks : most);
  if (a.rows) TB_SEQ_CUDA(seq_launch(kSeqNormBackward, (cudaStream_t)stream, launch_norm_backward, &n));
  TB_SEQ_CUDA(seq_launch(kSeqNormWeight, (cudaStream_t)stream, launch_norm_weight, &n));
  return TB_OK;
}

tb_status tb_rms_norm_backward(const tb_norm_backward_args* args, tb_stream stream) {
  return norm_backward_run("tb_rms_norm_backward", args, false, nullptr, stream);
}
int64_t tb_layer_norm_backward_workspace(int64_t rows, int32_t width) {
  return 2 * tb_rms_norm_backward_workspace(rows, width);
}
tb_status tb_layer_norm_backward(const tb_norm_backward_args* args, void* dbias, tb_stream stream) {
  return norm_backward_run("tb_layer_norm_backward", args, true, dbias, stream);
}

// Segment slots of a call, its walks along the rows: the segments of any offsets, or the grids.
static int64_t segment_slots(int64_t tokens, int32_t grids, int32_t segment) {
  return segment ? tokens / segment + grids : grids;
}

// -------------------------------------------------------------- convolution

static tb_status conv_sizes(const char* what, int64_t rows, int32_t channels, int32_t taps, int32_t type) {
  if (!type_ok(type)) return seq_fail(TB_ERR_INVALID_ARG, "%s: unknown type %d", what, type);
  if (rows < 0 || channels < 1) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad size", what);
  if (taps < 2 || taps > 4) return seq_fail(TB_ERR_INVALID_ARG, "%s: %d taps (2 to 4)", what, taps);
  if (rows > kMaxRows || up(channels, 128) * (rows + 1) > kMaxRows)
    return seq_fail(TB_ERR_TOO_LARGE, "%s: 2^31 rows, or blocks of 128 channels of them, or more", what);
  return TB_OK;
}
static tb_status conv_check(const char* what, const tb_conv_args& a) {
  const tb_status st = conv_sizes(what, a.tokens + (a.grids > 0 ? a.grids : 0), a.channels, a.taps, a.type);
  if (st != TB_OK) return st;
  if (a.tokens < 0 || a.grids < 0) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad size", what);
  if (!a.offsets && a.grids != 1) return seq_fail(TB_ERR_INVALID_ARG, "%s: %d grids without offsets", what, a.grids);
  if (a.grids == 0 && a.tokens) return seq_fail(TB_ERR_INVALID_ARG, "%s: tokens without grids", what);
  if (!a.weight || (a.tokens && !a.x)) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad pointer", what);
  return TB_OK;
}
// Rows that miss whole vectors go element by element: 60013 rows of 1028 channels
// in bf16 174 us, of 1024 53; with the gradient 279 and 138.
// Threads along the channels: up to 128 of a block, evenly over the blocks; rows
// of fewer share one.  Runs of rows are as long as gives every multiprocessor
// `threads` threads, within bounds.
static void conv_shape(ConvLaunch& l, int sms, int threads, int least, int most) {
  const int64_t cols = l.a.channels / l.vec;
  l.blocks_x = (int)up(cols, 128);
  l.per_x = (int)up(cols, l.blocks_x);
  l.threads = (int)up(128 / l.per_x * l.per_x, 32) * 32;
  const int64_t run = up(l.a.tokens * cols, (int64_t)threads * sms);
  l.run = (int)(run < least ? least : run > most ? most : run);
  l.runs = up(l.a.tokens, l.run);
}
static bool conv_fits(int vec, int size, const void* p, int64_t row) {
  return (uintptr_t)p % (vec * size) == 0 && row % vec == 0;
}

tb_status tb_causal_conv(const tb_conv_args* args, tb_stream stream) {
  const char* what = "tb_causal_conv";
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "%s: args is NULL", what);
  ConvLaunch l{};
  l.a = *args;
  const tb_conv_args& a = l.a;
  const tb_status st = conv_check(what, a);
  if (st != TB_OK) return st;
  if (a.tokens && !a.y) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad pointer", what);
  if (a.grids == 0 || (a.tokens == 0 && !a.state_out)) return TB_OK;
  const int sms = seq_sms();
  if (!sms) return seq_fail(TB_ERR_CUDA, "%s: no device", what);
  const int size = type_size(a.type), vec = 16 / size;
  const bool fits = a.channels % vec == 0 && conv_fits(vec, size, a.x, a.x_row) && conv_fits(vec, size, a.y, a.y_row) &&
                    aligned16(a.state) && aligned16(a.state_out) && aligned16(a.weight) && aligned16(a.bias);
  l.vec = fits ? vec : 1;
  conv_shape(l, sms, 384, 4, 512);
  TB_SEQ_CUDA(seq_launch(kSeqConv, (cudaStream_t)stream, launch_conv, &l));
  return TB_OK;
}

// Threads a multiprocessor that a wave of runs is cut for.  Registers (124 in 16
// bits, 92 in 32) would hold 512 and 640.
constexpr int kConvBackThreads = 384, kConvBackLeast = 8, kConvBackMost = 512;

int64_t tb_causal_conv_backward_workspace(int64_t tokens, int32_t channels, int32_t taps) {
  if (tokens < 0 || channels < 1 || taps < 2 || taps > 4) return 0;
  const int sms = seq_sms();
  int64_t most = 0;
  for (int vec = 1; vec <= 4; vec *= 2) {
    if (channels % vec) continue;
    ConvLaunch l{};
    l.a.tokens = tokens, l.a.channels = channels, l.vec = vec;
    conv_shape(l, sms ? sms : 256, kConvBackThreads, kConvBackLeast, kConvBackMost);
    const int64_t parts = up(l.runs, l.threads / l.per_x);
    if (parts > most) most = parts;
  }
  return most * (taps + 1) * channels * (int64_t)sizeof(float);
}

tb_status tb_causal_conv_backward(const tb_conv_backward_args* args, tb_stream stream) {
  const char* what = "tb_causal_conv_backward";
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "%s: args is NULL", what);
  ConvBackwardLaunch l{};
  l.f.a = args->f;
  l.g = *args;
  const tb_conv_args& a = l.f.a;
  const tb_conv_backward_args& g = l.g;
  const tb_status st = conv_check(what, a);
  if (st != TB_OK) return st;
  if (!g.dweight || (a.tokens && (!g.dy || !g.dx || !g.workspace))) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad pointer", what);
  const int sms = seq_sms();
  if (!sms) return seq_fail(TB_ERR_CUDA, "%s: no device", what);
  const int64_t need = tb_causal_conv_backward_workspace(a.tokens, a.channels, a.taps);
  if (g.workspace_bytes < need || !aligned16(g.workspace))
    return seq_fail(TB_ERR_INVALID_ARG, "%s: a workspace of %lld bytes, %lld needed", what, (long long)g.workspace_bytes,
                    (long long)need);
  // vectors of 8 bytes: the windows of x and of its gradient take twice the registers of the forward pass
  const int size = type_size(a.type), vec = 8 / size;
  const bool fits = a.channels % vec == 0 && conv_fits(vec, size, a.x, a.x_row) && conv_fits(vec, size, g.dy, g.dy_row) &&
                    conv_fits(vec, size, g.dx, g.dx_row) && conv_fits(vec, size, a.state, 0) &&
                    conv_fits(vec, size, g.dstate_out, 0) && conv_fits(vec, size, g.dstate, 0) && conv_fits(vec, size, a.weight, 0) &&
                    conv_fits(vec, size, a.bias, 0);
  l.f.vec = fits ? vec : 1;
  conv_shape(l.f, sms, kConvBackThreads, kConvBackLeast, kConvBackMost);
  l.parts = up(l.f.runs, l.f.threads / l.f.per_x);
  if (a.tokens || (g.dstate && a.grids)) TB_SEQ_CUDA(seq_launch(kSeqConvBackward, (cudaStream_t)stream, launch_conv_backward, &l));
  TB_SEQ_CUDA(seq_launch(kSeqConvWeight, (cudaStream_t)stream, launch_conv_weight, &l));
  return TB_OK;
}

tb_status tb_causal_conv_step(const tb_conv_step_args* args, tb_stream stream) {
  const char* what = "tb_causal_conv_step";
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "%s: args is NULL", what);
  ConvStepLaunch l{};
  l.a = *args;
  const tb_conv_step_args& a = l.a;
  const tb_status st = conv_sizes(what, a.streams, a.channels, a.taps, a.type);
  if (st != TB_OK) return st;
  if (a.num_slots < 0) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad size", what);
  if (a.streams == 0) return TB_OK;
  if (!a.slots && a.num_slots < a.streams)
    return seq_fail(TB_ERR_INVALID_ARG, "%s: %lld streams, %lld states", what, (long long)a.streams, (long long)a.num_slots);
  if (!a.x || !a.weight || !a.y || (a.num_slots && !a.state)) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad pointer", what);
  const int size = type_size(a.type), vec = 16 / size;
  const bool fits = a.channels % vec == 0 && conv_fits(vec, size, a.x, a.x_row) && conv_fits(vec, size, a.y, a.y_row) &&
                    aligned16(a.state) && aligned16(a.weight) && aligned16(a.bias);
  l.vec = fits ? vec : 1;
  TB_SEQ_CUDA(seq_launch(kSeqConvStep, (cudaStream_t)stream, launch_conv_step, &l));
  return TB_OK;
}

// ----------------------------------------------------------- selective scan

// Channels in the workspace: each group's rounded up to whole tiles.
static int64_t scan_wide(int32_t channels, int32_t groups) { return up(channels / groups, kScanChannels) * kScanChannels * groups; }

// Tiles of kScanChannels channels and blocks of states; four warps of tiles a
// block, fewer where their states would not fit in shared memory.
static void scan_shape(ScanLaunch& l, int32_t channels, int32_t states, int32_t groups) {
  l.group_tiles = (int32_t)up(channels / groups, kScanChannels);
  l.group_pad = l.group_tiles * kScanChannels;
  l.wide = l.group_pad * groups;
  l.pass = states <= 8 ? 8 : 16;
  l.pad = (int32_t)up(states, l.pass) * l.pass;
  l.warps = l.pad <= 32 ? 4 : l.pad <= 128 ? 2 : 1;
  l.blocks_x = (int32_t)up((int64_t)groups * l.group_tiles, l.warps);
}

// Rows of a segment of the forward pass, 0: grids are walked whole.  A walk is
// sequential along a grid and a warp's, so a call with few of them is split, so
// that four blocks a multiprocessor run at once; the segments' own states cost
// most of a walk once more (66300 rows of 2048 channels: one grid, split, 1.12 ms;
// 64 of 1035 rows each, whole, 0.78).  The rule knows how many grids there are and
// not how long: one of 60000 rows among 63 of 100 is one warp's walk for each 64
// channels and takes 28 ms.
static int32_t scan_segment(const ScanLaunch& l, int64_t tokens, int32_t grids, int sms) {
  const int64_t blocks = (int64_t)grids * l.blocks_x;
  if (grids <= 0 || blocks >= 3ll * sms || tokens < 96ll * grids) return 0;
  const int64_t slots = 4ll * sms / l.blocks_x - grids;
  int64_t seg = up(up(tokens, slots > 1 ? slots : 1), kTileRows) * kTileRows;
  if (seg < 32) seg = 32;
  return tokens >= 2 * seg * grids ? (int32_t)seg : 0;
}

struct ScanCarve {
  int64_t seg, sum, tile, tile_sum, seg_back, bc, part_a, part_d, acc, bytes;
  int32_t quads, runs, per_run;
};
static ScanCarve scan_carve(int64_t slots, int64_t tokens, int32_t channels, int32_t groups, const ScanLaunch& l, bool backward,
                            int sms) {
  ScanCarve c{};
  auto take = [&](int64_t floats) {
    const int64_t at = c.bytes;
    c.bytes += up(floats * 4, 256) * 256;
    return at;
  };
  c.seg = take(slots * l.wide * l.pad);
  c.sum = take(slots * l.wide);
  if (!backward) return c;
  c.tile = take(tokens / kTileRows * l.wide * l.pad);
  c.tile_sum = take(tokens / kTileRows * l.wide);
  c.quads = (int32_t)up(channels / groups, 128);
  // blocks take runs of chunks, whose parts of da they keep in registers: as many as make six waves or so
  const int64_t blocks = slots * groups * c.quads;
  c.per_run = (int32_t)up(blocks, 12ll * sms);
  c.runs = (int32_t)up(slots, c.per_run > 0 ? c.per_run : 1);
  c.seg_back = take(slots * l.wide * l.pad);
  c.bc = take((int64_t)c.quads * tokens * groups * 2 * l.pad);
  c.part_a = take((int64_t)c.runs * l.wide * l.pad);
  c.part_d = take((int64_t)c.runs * 2 * l.wide);
  if (l.pad > l.pass) c.acc = take(tokens * channels * 3);
  return c;
}

// Rows of a chunk of the gradient: shorter ones where two blocks a
// multiprocessor would not run.
static int32_t scan_chunk(const ScanLaunch& l, int64_t tokens, int32_t groups, int sms) {
  int32_t chunk = 64;
  while (chunk > 16 && tokens / chunk * groups * up(l.group_pad, 128) < 2ll * sms) chunk /= 2;
  return chunk;
}

int64_t tb_selective_scan_workspace(int64_t tokens, int32_t grids, int32_t channels, int32_t states, int32_t groups,
                                    int32_t backward) {
  if (tokens < 0 || grids < 0 || channels < 1 || states < 1 || states > 256 || groups < 1 || channels % groups) return 0;
  if (tokens > kMaxRows || scan_wide(channels, groups) > kMaxRows) return 0;  // refused by the call
  ScanLaunch l{};
  scan_shape(l, channels, states, groups);
  int sms = seq_sms();
  if (!sms) sms = 256;
  l.segment = backward ? scan_chunk(l, tokens, groups, sms) : scan_segment(l, tokens, grids, sms);
  if (!l.segment) return 0;
  return scan_carve(segment_slots(tokens, grids, l.segment), tokens, channels, groups, l, backward, sms).bytes;
}

static tb_status scan_sizes(const char* what, int64_t rows, int32_t channels, int32_t states, int32_t groups, int32_t type) {
  if (!type_ok(type)) return seq_fail(TB_ERR_INVALID_ARG, "%s: unknown type %d", what, type);
  if (rows < 0 || channels < 1 || states < 1 || groups < 1 || channels % groups)
    return seq_fail(TB_ERR_INVALID_ARG, "%s: bad size (%d channels in %d groups)", what, channels, groups);
  if (states > 256 || rows > kMaxRows)
    return seq_fail(TB_ERR_TOO_LARGE, "%s: %d states a channel (at most 256), or 2^31 rows", what, states);
  return TB_OK;
}

// Completes l for its l.a: the walk, and the carve of a workspace of a.workspace_bytes.
static tb_status scan_plan(const char* what, ScanLaunch& l, bool backward, ScanCarve& c, int sms) {
  const tb_scan_args& a = l.a;
  const int size = type_size(a.type);
  scan_shape(l, a.channels, a.states, a.groups);
  l.offsets = a.offsets, l.tokens = a.tokens, l.grids = a.grids;
  l.segment = backward ? scan_chunk(l, a.tokens, a.groups, sms) : scan_segment(l, a.tokens, a.grids, sms);
  const int64_t slots = segment_slots(a.tokens, a.grids, l.segment);
  const int64_t per_slot = (int64_t)a.groups * l.group_tiles;
  const int64_t join = up((int64_t)l.wide * (l.pad / 4), 128);
  if (slots > kMaxRows / per_slot || a.grids > kMaxRows / join ||
      (backward && a.tokens > kMaxRows / (up((int64_t)a.groups * 2 * a.states, 512) + 1) - join * 32))
    return seq_fail(TB_ERR_TOO_LARGE, "%s: 2^31 blocks or more", what);
  l.segments = (int32_t)slots;
  auto whole_rows = [&](const void* p, int64_t row) { return !p || (aligned16(p) && whole(row, size)); };
  l.vec = whole_rows(a.x, a.x_row) && whole_rows(a.dt, a.dt_row) && whole_rows(a.z, a.z_row) &&
          (a.groups == 1 || whole(a.channels / a.groups, size));
  if (!l.segment) return TB_OK;
  c = scan_carve(slots, a.tokens, a.channels, a.groups, l, backward, sms);
  if (c.bytes && (!a.workspace || a.workspace_bytes < c.bytes || ((uintptr_t)a.workspace & 255)))
    return seq_fail(TB_ERR_INVALID_ARG, "%s: a workspace of %lld bytes, %lld needed", what, (long long)a.workspace_bytes,
                    (long long)c.bytes);
  l.seg = (float*)((char*)a.workspace + c.seg);
  l.sum = (float*)((char*)a.workspace + c.sum);
  if (backward) {
    l.tile = (float*)((char*)a.workspace + c.tile);
    l.tile_sum = (float*)((char*)a.workspace + c.tile_sum);
  }
  return TB_OK;
}

static tb_status scan_check(const char* what, const tb_scan_args& a) {
  const tb_status st = scan_sizes(what, a.tokens, a.channels, a.states, a.groups, a.type);
  if (st != TB_OK) return st;
  if (a.grids < 0) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad size", what);
  if (!a.offsets && a.grids != 1) return seq_fail(TB_ERR_INVALID_ARG, "%s: %d grids without offsets", what, a.grids);
  if (a.grids == 0 && a.tokens) return seq_fail(TB_ERR_INVALID_ARG, "%s: tokens without grids", what);
  if (!a.a || (a.tokens && (!a.x || !a.dt || !a.b || !a.c))) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad pointer", what);
  if (scan_wide(a.channels, a.groups) > kMaxRows)
    return seq_fail(TB_ERR_TOO_LARGE, "%s: 2^31 channels or more, each group's rounded up to %d", what, kScanChannels);
  return TB_OK;
}

tb_status tb_selective_scan(const tb_scan_args* args, tb_stream stream) {
  const char* what = "tb_selective_scan";
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "%s: args is NULL", what);
  ScanLaunch l{};
  l.a = *args;
  const tb_scan_args& a = l.a;
  tb_status st = scan_check(what, a);
  if (st != TB_OK) return st;
  if (a.tokens && !a.y) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad pointer", what);
  if (a.grids == 0 || (a.tokens == 0 && !a.state_out)) return TB_OK;
  const int sms = seq_sms();
  if (!sms) return seq_fail(TB_ERR_CUDA, "%s: no device", what);
  ScanCarve c{};
  st = scan_plan(what, l, false, c, sms);
  if (st != TB_OK) return st;
  if (l.segment) {
    TB_SEQ_CUDA(seq_launch(kSeqSelectiveStates, (cudaStream_t)stream, launch_scan_states, &l));
    TB_SEQ_CUDA(seq_launch(kSeqSelectiveJoin, (cudaStream_t)stream, launch_scan_join, &l));
  }
  TB_SEQ_CUDA(seq_launch(kSeqSelective, (cudaStream_t)stream, launch_scan, &l));
  return TB_OK;
}

tb_status tb_selective_scan_backward(const tb_scan_backward_args* args, tb_stream stream) {
  const char* what = "tb_selective_scan_backward";
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "%s: args is NULL", what);
  ScanBackwardLaunch g{};
  g.f.a = args->f;
  g.g = *args;
  const tb_scan_args& a = g.f.a;
  tb_status st = scan_check(what, a);
  if (st != TB_OK) return st;
  if (!g.g.da || (a.tokens && (!g.g.dy || !g.g.dx || !g.g.ddt || !g.g.db || !g.g.dc || (a.z && !g.g.dz))))
    return seq_fail(TB_ERR_INVALID_ARG, "%s: bad pointer", what);
  const int sms = seq_sms();
  if (!sms) return seq_fail(TB_ERR_CUDA, "%s: no device", what);
  ScanCarve c{};
  st = scan_plan(what, g.f, true, c, sms);
  if (st != TB_OK) return st;
  g.f.vec = g.f.vec && (!g.g.dy || (aligned16(g.g.dy) && whole(g.g.dy_row, type_size(a.type))));
  char* const work = (char*)a.workspace;
  g.seg_back = (float*)(work + c.seg_back);
  g.bc = (float*)(work + c.bc);
  g.part_a = (float*)(work + c.part_a);
  g.part_d = (float*)(work + c.part_d);
  g.acc = c.acc ? (float*)(work + c.acc) : nullptr;
  g.quads = c.quads, g.runs = c.runs, g.per_run = c.per_run;
  const cudaStream_t s = (cudaStream_t)stream;
  if (a.grids) {
    TB_SEQ_CUDA(seq_launch(kSeqSelectiveStates, s, launch_scan_states, &g.f));
    TB_SEQ_CUDA(seq_launch(kSeqSelectiveStates, s, launch_scan_carry, &g));
    TB_SEQ_CUDA(seq_launch(kSeqSelectiveJoin, s, launch_scan_back_join, &g));
    TB_SEQ_CUDA(seq_launch(kSeqSelectiveBackward, s, launch_scan_backward, &g));
  }
  TB_SEQ_CUDA(seq_launch(kSeqSelectiveSums, s, launch_scan_sums, &g));
  return TB_OK;
}

tb_status tb_selective_scan_step(const tb_scan_step_args* args, tb_stream stream) {
  const char* what = "tb_selective_scan_step";
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "%s: args is NULL", what);
  ScanStepLaunch l{};
  l.a = *args;
  const tb_scan_step_args& a = l.a;
  const tb_status st = scan_sizes(what, a.streams, a.channels, a.states, a.groups, a.type);
  if (st != TB_OK) return st;
  if (a.num_slots < 0) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad size", what);
  if (a.streams == 0) return TB_OK;
  if (!a.slots && a.num_slots < a.streams)
    return seq_fail(TB_ERR_INVALID_ARG, "%s: %lld streams, %lld states", what, (long long)a.streams, (long long)a.num_slots);
  if (!a.x || !a.dt || !a.a || !a.b || !a.c || !a.y ||
      (a.num_slots && (!a.state || (uintptr_t)a.state % (a.states % 4 == 0 ? 16 : 4))))
    return seq_fail(TB_ERR_INVALID_ARG, "%s: bad pointer (states are 16-byte aligned where they are a multiple of 4)", what);
  const int sms = seq_sms();
  if (!sms) return seq_fail(TB_ERR_CUDA, "%s: no device", what);
  const int size = type_size(a.type);
  auto fours = [&](const void* p, int64_t row, int64_t group) {
    return (uintptr_t)p % (4 * size) == 0 && row % 4 == 0 && (a.groups == 1 || group % 4 == 0);
  };
  l.vec = a.states % 4 == 0 && a.states <= 16 && aligned16(a.a) && aligned16(a.state) && fours(a.b, a.b_row, a.b_group) &&
          fours(a.c, a.c_row, a.c_group);
  // fours of streams, several a block while there are blocks enough: its rates stay in registers
  const int64_t blocks_x = up(a.channels, 32), fours_of = a.streams * blocks_x / (32ll * sms);
  l.per_block = 4 * (int)(fours_of < 1 ? 1 : fours_of > 4 ? 4 : fours_of);
  if (blocks_x > kMaxRows / a.streams) return seq_fail(TB_ERR_TOO_LARGE, "%s: 2^31 blocks or more", what);
  TB_SEQ_CUDA(seq_launch(kSeqSelectiveStep, (cudaStream_t)stream, launch_scan_step, &l));
  return TB_OK;
}

// --------------------------------------------------------- linear attention

struct LinSizes {
  int64_t tokens;
  int32_t grids, heads, key, value, type;
};

// Tokens of a segment, 0: grids are walked whole.  A walk is sequential along
// a grid, so a call with few grids and heads is split along the rows: the
// segments' own states first, their joining, then the outputs.  One block of a
// chunk kernel (of two heads, where they are small) runs on a multiprocessor;
// the states pass is as long as a walk nearly, and the two more launches take
// 6 us.  So it pays where whole grids leave more than half the
// multiprocessors idle (10 grids of 3000 rows and 6 heads, 60 walks: 85 us
// split, 72 whole; 16 unequal grids, 64 walks: 164 and 275), and where a grid
// is several segments (one grid of 600 rows: 18.6 us whole, 16.5 split; 4 of 600
// with 4 heads of 128: 18.6 and 20.6).  Long grids leave up to a third idle (8
// grids of 7500 rows, the gradient of 4 heads of 128, 96 walks: 217 us split,
// 254 whole; of 2500: 106 and 89), less long ones where the chunk is slowest
// (14 of 1400 in fp16, the gradient of 2 heads of 96 x 128, 84 walks: 143 and
// 238).
// Segments are as short as gives each multiprocessor one, the chain being what
// costs (in fp32 one grid of 1000 rows and 4 heads: 20.6 us by 64 rows, 34.9 by
// 256; 5 unequal ones, 1333 rows, 20.6 split so, 41 whole), but in bf16 two
// chunks (one grid of 2000 rows, 4 heads of 128: 20.6 us by 128 rows, 26.3 by
// 64); where that takes more than 256 rows, two a multiprocessor.
static int32_t segment_tokens(const LinSizes& z, int problems, int sms) {
  const bool tc = z.type == TB_TYPE_BF16, pairs = tc && linear_pairs(z.key, z.value);
  const int64_t walks = (int64_t)(pairs ? (z.heads + 1) / 2 : z.heads) * problems;
  const bool slow = !tc && (z.key > 64 || z.value > 64), lengthy = z.tokens >= (slow ? 1024ll : 4096ll) * z.grids;
  if (z.grids <= 0 || 20ll * z.grids * walks > (lengthy ? 14ll : 9ll) * sms) return 0;
  int64_t seg = up(up(z.tokens * walks, sms - z.grids * walks), 64) * 64;
  if (seg > 256) {
    seg = up(up(z.tokens * walks, 2 * sms), 64) * 64;
    if (seg < 256) seg = 256;
  }
  if (tc && seg < 128) seg = 128;
  const int64_t least = tc ? (seg < 256 ? 768 : 3 * seg) : seg < 96 ? 192 : 2 * seg;
  return z.tokens >= least * z.grids ? (int32_t)seg : 0;
}

int64_t tb_linear_attention_workspace(int64_t tokens, int32_t grids, int32_t heads, int32_t key, int32_t value,
                                      int32_t type, int32_t backward) {
  if (tokens < 0 || grids < 0 || heads < 1 || key < 1 || value < 1) return 0;
  const int sms = seq_sms();
  const int problems = backward ? 3 : 1;
  const int32_t seg = segment_tokens({tokens, grids, heads, key, value, type}, problems, sms ? sms : 256);
  return seg ? segment_slots(tokens, grids, seg) * heads * key * value * 4 * problems : 0;
}

static tb_status linear_check(const char* what, const tb_linear_args& a) {
  if (!type_ok(a.type)) return seq_fail(TB_ERR_INVALID_ARG, "%s: unknown type %d", what, a.type);
  if (a.tokens < 0 || a.grids < 0 || a.heads < 1 || a.key < 1 || a.value < 1)
    return seq_fail(TB_ERR_INVALID_ARG, "%s: bad size", what);
  if (a.key > 128 || a.value > 128)
    return seq_fail(TB_ERR_TOO_LARGE, "%s: heads of %d keys and %d values (at most 128)", what, a.key, a.value);
  if (a.tokens > kMaxRows || a.heads > 65535 || (int64_t)a.grids * a.heads > kMaxRows)
    return seq_fail(TB_ERR_TOO_LARGE, "%s: 2^31 tokens, 65536 heads or 2^31 states, or more", what);
  if (!a.offsets && a.grids != 1) return seq_fail(TB_ERR_INVALID_ARG, "%s: %d grids without offsets", what, a.grids);
  if (a.grids == 0 && a.tokens) return seq_fail(TB_ERR_INVALID_ARG, "%s: tokens without grids", what);
  if ((a.tokens && (!a.q || !a.k || !a.v)) || !a.decay) return seq_fail(TB_ERR_INVALID_ARG, "%s: bad pointer", what);
  return TB_OK;
}

static tb_status linear_run(const char* what, const tb_linear_args& a, ChunkLaunch& g, cudaStream_t s) {
  LinLaunch& l = g.l;
  const int sms = seq_sms();
  if (!sms) return seq_fail(TB_ERR_CUDA, "%s: no device", what);
  l.type = a.type;
  l.heads = a.heads;
  l.grids = a.grids;
  l.tokens = a.tokens;
  l.offsets = a.offsets;
  l.decay = a.decay;
  l.segment = segment_tokens({a.tokens, a.grids, a.heads, a.key, a.value, a.type}, l.n, sms);
  const int64_t slots = segment_slots(a.tokens, a.grids, l.segment);
  if (slots * a.heads * l.n > kMaxRows) return seq_fail(TB_ERR_TOO_LARGE, "%s: 2^31 walks or more", what);
  l.segments = (int32_t)slots;
  if (l.segment) {
    const int64_t one = slots * a.heads * a.key * a.value;
    if (!a.workspace || a.workspace_bytes < one * 4 * l.n || ((uintptr_t)a.workspace & 255))
      return seq_fail(TB_ERR_INVALID_ARG, "%s: a workspace of %lld bytes, %lld needed", what,
                      (long long)a.workspace_bytes, (long long)(one * 4 * l.n));
    for (int i = 0; i < l.n; ++i) l.p[i].seg = (float*)a.workspace + i * one;
  }
  // A chunk of 64 rows costs the tensor cores the same with one row in it: short grids take the recurrence (512 grids, 8
  // heads of 128 x 128, us: 15 rows in bf16 167, 16 by chunks 149; 24 rows in fp16 267, 270 by chunks, in fp32 271 and 315).
  const bool longer = a.tokens >= (a.type == TB_TYPE_BF16 ? 16ll : 24ll) * a.grids;
  const bool chunks = longer && linear_chunk_plan(g);
  for (int i = 0; i < l.n; ++i) {
    LinProblem& p = l.p[i];
    const int size = type_size(a.type);
    p.vec = p.K % 8 == 0 ? (aligned16(p.a) && whole(p.a_row, size) && whole(p.a_head, size) ? 1 : 0) |
                               (aligned16(p.b) && whole(p.b_row, size) && whole(p.b_head, size) ? 2 : 0)
                         : 0;
  }
  l.phase = 0;
  // With more walks than multiprocessors the last to start should be short ones.
  l.sorted = !l.segment && a.grids > 1 && a.grids <= kLinMaxSorted && (int64_t)a.grids * a.heads * l.n > sms;
  if (l.segment) {
    l.phase = 1;  // of grids of 192 rows and more on average: never the recurrence
    if (chunks) TB_SEQ_CUDA(seq_launch(kSeqChunkStates, s, launch_linear_chunks, &g));
    else TB_SEQ_CUDA(seq_launch(kSeqSplitStates, s, launch_linear_split, &l));
    TB_SEQ_CUDA(seq_launch(kSeqCombine, s, launch_linear_combine, &l));
    l.phase = 2;
  }
  if (chunks) TB_SEQ_CUDA(seq_launch(kSeqChunks, s, launch_linear_chunks, &g));
  else if (longer) TB_SEQ_CUDA(seq_launch(kSeqSplit, s, launch_linear_split, &l));
  else TB_SEQ_CUDA(seq_launch(kSeqScan, s, launch_linear_scan, &l));
  return TB_OK;
}

tb_status tb_linear_attention(const tb_linear_args* args, tb_stream stream) {
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "tb_linear_attention: args is NULL");
  const tb_linear_args& a = *args;
  const tb_status st = linear_check("tb_linear_attention", a);
  if (st != TB_OK) return st;
  if (a.tokens && !a.out) return seq_fail(TB_ERR_INVALID_ARG, "tb_linear_attention: bad pointer");
  if (a.grids == 0 || (a.tokens == 0 && !a.state_out)) return TB_OK;
  ChunkLaunch g;
  memset(&g, 0, sizeof g);
  LinLaunch& l = g.l;
  l.n = 1;
  LinProblem& p = l.p[0];
  p.a = a.q, p.a_row = a.q_row, p.a_head = a.q_head;
  p.b = a.k, p.b_row = a.k_row, p.b_head = a.k_head;
  p.c = a.v, p.c_row = a.v_row, p.c_head = a.v_head;
  p.out = a.out, p.o_row = a.out_row, p.o_head = a.out_head;
  p.K = a.key, p.V = a.value;
  p.first = a.state, p.first_k = a.value, p.first_v = 1;
  p.last = a.state_out;
  p.mul = a.scale, p.fold = 1.f;
  return linear_run("tb_linear_attention", a, g, (cudaStream_t)stream);
}

tb_status tb_linear_attention_backward(const tb_linear_backward_args* args, tb_stream stream) {
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "tb_linear_attention_backward: args is NULL");
  const tb_linear_args& a = args->f;
  const tb_linear_backward_args& g = *args;
  const tb_status st = linear_check("tb_linear_attention_backward", a);
  if (st != TB_OK) return st;
  if (a.tokens && (!g.grad || !g.dq || !g.dk || !g.dv))
    return seq_fail(TB_ERR_INVALID_ARG, "tb_linear_attention_backward: bad pointer");
  if (a.grids == 0 || (a.tokens == 0 && !g.dstate)) return TB_OK;
  ChunkLaunch plan;
  memset(&plan, 0, sizeof plan);
  LinLaunch& l = plan.l;
  l.n = 3;
  {  // dv, with the state U and its end, the gradient of the first state
    LinProblem& p = l.p[0];
    p.a = a.k, p.a_row = a.k_row, p.a_head = a.k_head;
    p.b = a.q, p.b_row = a.q_row, p.b_head = a.q_head;
    p.c = g.grad, p.c_row = g.grad_row, p.c_head = g.grad_head;
    p.out = g.dv, p.o_row = g.dv_row, p.o_head = g.dv_head;
    p.K = a.key, p.V = a.value;
    p.first = g.dstate_out, p.first_k = a.value, p.first_v = 1;
    p.last = g.dstate;
    p.mul = 1.f, p.fold = a.scale;
    p.reverse = p.late = 1;
  }
  {  // dk, with U^T
    LinProblem& p = l.p[1];
    p.a = a.v, p.a_row = a.v_row, p.a_head = a.v_head;
    p.b = g.grad, p.b_row = g.grad_row, p.b_head = g.grad_head;
    p.c = a.q, p.c_row = a.q_row, p.c_head = a.q_head;
    p.out = g.dk, p.o_row = g.dk_row, p.o_head = g.dk_head;
    p.K = a.value, p.V = a.key;
    p.first = g.dstate_out, p.first_k = 1, p.first_v = a.value;
    p.mul = 1.f, p.fold = a.scale;
    p.reverse = p.late = 1;
  }
  {  // dq, with S^T
    LinProblem& p = l.p[2];
    p.a = g.grad, p.a_row = g.grad_row, p.a_head = g.grad_head;
    p.b = a.v, p.b_row = a.v_row, p.b_head = a.v_head;
    p.c = a.k, p.c_row = a.k_row, p.c_head = a.k_head;
    p.out = g.dq, p.o_row = g.dq_row, p.o_head = g.dq_head;
    p.K = a.value, p.V = a.key;
    p.first = a.state, p.first_k = 1, p.first_v = a.value;
    p.mul = a.scale, p.fold = 1.f;
  }
  return linear_run("tb_linear_attention_backward", a, plan, (cudaStream_t)stream);
}

tb_status tb_linear_attention_status(tb_stream stream) {
  int dev = 0;
  unsigned int chunks = 0, split = 0;
  TB_SEQ_CUDA(cudaGetDevice(&dev));
  TB_SEQ_CUDA(linear_gave_up((cudaStream_t)stream, &chunks));
  TB_SEQ_CUDA(linear_split_gave_up((cudaStream_t)stream, &split));
  bool news = false;
  try {
    static std::mutex lock;
    static std::map<std::pair<int, tb_stream>, unsigned int> seen;  // of each stream's last call
    const std::lock_guard<std::mutex> guard(lock);
    unsigned int& last = seen[{dev, stream}];
    news = (int)(chunks + split - last) > 0;
    if (news) last = chunks + split;
  } catch (...) {
    return seq_fail(TB_ERR_OOM, "tb_linear_attention_status: out of host memory");
  }
  if (news) return seq_fail(TB_ERR_DEVICE_TIMEOUT, "tb_linear_attention: a device-side wait timed out");
  return TB_OK;
}

tb_status tb_linear_attention_selftest_wait(int32_t kernel, int32_t spin_limit, tb_stream stream) {
  if (kernel < 0 || kernel > 1 || spin_limit < 1 || spin_limit > 1 << 22)
    return seq_fail(TB_ERR_INVALID_ARG, "tb_linear_attention_selftest_wait: kernel %d, %d polls", kernel, spin_limit);
  const uint32_t polls = (uint32_t)spin_limit;
  TB_SEQ_CUDA(seq_launch(kSeqSelftest, (cudaStream_t)stream, kernel ? linear_split_selftest : linear_selftest, &polls));
  return TB_OK;
}

tb_status tb_linear_attention_step(const tb_linear_step_args* args, tb_stream stream) {
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "tb_linear_attention_step: args is NULL");
  StepLaunch l;
  l.a = *args;
  const tb_linear_step_args& a = l.a;
  if (!type_ok(a.type)) return seq_fail(TB_ERR_INVALID_ARG, "tb_linear_attention_step: unknown type %d", a.type);
  if (a.streams < 0 || a.num_slots < 0 || a.heads < 1 || a.key < 1 || a.value < 1)
    return seq_fail(TB_ERR_INVALID_ARG, "tb_linear_attention_step: bad size");
  if (a.key > 256 || a.value > 256 || a.streams * a.heads > kMaxRows)
    return seq_fail(TB_ERR_TOO_LARGE, "tb_linear_attention_step: heads of %d keys and %d values (at most 256), or 2^31 states",
                    a.key, a.value);
  if (a.streams == 0) return TB_OK;
  if (!a.slots && a.num_slots < a.streams)
    return seq_fail(TB_ERR_INVALID_ARG, "tb_linear_attention_step: %lld streams, %lld states", (long long)a.streams,
                    (long long)a.num_slots);
  // states of whole vectors are read by vectors, others element by element
  if (!a.q || !a.k || !a.v || !a.out || !a.decay ||
      (a.num_slots && (!a.state || (uintptr_t)a.state % (a.value % 4 == 0 ? 16 : 4))))
    return seq_fail(TB_ERR_INVALID_ARG, "tb_linear_attention_step: bad pointer (states are 16-byte aligned where the values "
                    "of a head are a multiple of 4)");
  TB_SEQ_CUDA(seq_launch(kSeqStep, (cudaStream_t)stream, launch_linear_step, &l));
  return TB_OK;
}

}  // extern "C"
