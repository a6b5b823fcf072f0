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

tb_status tb_rms_norm(const tb_norm_args* args, tb_stream stream) {
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "tb_rms_norm: args is NULL");
  NormLaunch n;
  n.a = *args;
  tb_norm_args& a = n.a;
  if (!type_ok(a.type)) return seq_fail(TB_ERR_INVALID_ARG, "tb_rms_norm: unknown type %d", a.type);
  if (a.rows < 0 || a.width < 1) return seq_fail(TB_ERR_INVALID_ARG, "tb_rms_norm: bad size");
  if (a.width > 16384 || a.rows > kMaxRows)
    return seq_fail(TB_ERR_TOO_LARGE, "tb_rms_norm: rows of %d elements (at most 16384), or 2^31 rows", a.width);
  if (a.rows == 0) return TB_OK;
  if (!a.x || !a.weight || !a.y || (a.h_out && !a.residual) || (a.fp8 != 0) != (a.scale != nullptr))
    return seq_fail(TB_ERR_INVALID_ARG, "tb_rms_norm: bad pointer");
  const int sms = seq_sms();
  if (!sms) return seq_fail(TB_ERR_CUDA, "tb_rms_norm: no device");
  const int size = type_size(a.type), vec = 16 / size;
  n.vec = a.width % vec == 0 && aligned16(a.x) && aligned16(a.weight) && whole(a.x_row, size);
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

tb_status tb_rms_norm_backward(const tb_norm_backward_args* args, tb_stream stream) {
  if (!args) return seq_fail(TB_ERR_INVALID_ARG, "tb_rms_norm_backward: args is NULL");
  NormBackwardLaunch n;
  n.a = *args;
  tb_norm_backward_args& a = n.a;
  if (!type_ok(a.type)) return seq_fail(TB_ERR_INVALID_ARG, "tb_rms_norm_backward: unknown type %d", a.type);
  if (a.rows < 0 || a.width < 1) return seq_fail(TB_ERR_INVALID_ARG, "tb_rms_norm_backward: bad size");
  if (a.width > 16384 || a.rows > kMaxRows)
    return seq_fail(TB_ERR_TOO_LARGE, "tb_rms_norm_backward: rows of %d elements (at most 16384), or 2^31 rows", a.width);
  if (!a.dweight || (a.rows && (!a.dy || !a.h || !a.weight || !a.dx || !a.workspace)))
    return seq_fail(TB_ERR_INVALID_ARG, "tb_rms_norm_backward: bad pointer");
  const int sms = seq_sms();
  if (!sms) return seq_fail(TB_ERR_CUDA, "tb_rms_norm_backward: no device");
  const int64_t most = norm_backward_blocks(a.rows, sms);
  if (a.workspace_bytes < most * a.width * (int64_t)sizeof(float) || !aligned16(a.workspace))
    return seq_fail(TB_ERR_INVALID_ARG, "tb_rms_norm_backward: a workspace of %lld bytes, %lld needed",
                    (long long)a.workspace_bytes, (long long)(most * a.width * 4));
  const int size = type_size(a.type), vec = 16 / size;
  n.vec = a.width % vec == 0 && aligned16(a.dy) && aligned16(a.h) && aligned16(a.weight) && aligned16(a.dx) &&
          whole(a.dy_row, size) && whole(a.h_row, size) && whole(a.dx_row, size);
  if (a.dh) n.vec = n.vec && aligned16(a.dh) && whole(a.dh_row, size);
  const bool many = a.rows >= 4ll * sms;
  const int tensors = a.dh ? 3 : 2;
  const bool dense = aligned16(a.dy) && aligned16(a.h) && aligned16(a.dx) && a.dy_row == a.width && a.h_row == a.width &&
                     a.dx_row == a.width && (!a.dh || (aligned16(a.dh) && a.dh_row == a.width));
  const NormGroups groups = !n.vec && (many || a.width > 4096) && dense ? norm_groups(a.width, size, tensors, 8) : NormGroups{0, 0};
  int64_t blocks;
  n.groups = groups.rows > 0;
  if (n.groups) {
    n.nv = groups.stages;
    n.rows = groups.rows;
    blocks = norm_group_blocks(a.rows, a.width, size, tensors, groups, 8, sms, &n.per_row);
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

static int64_t segment_slots(int64_t tokens, int32_t grids, int32_t segment) {
  return segment ? tokens / segment + grids : grids;
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
