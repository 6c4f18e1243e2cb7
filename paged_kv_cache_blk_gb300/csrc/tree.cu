// Entry points of the tree decode and the windowed prefill (pkv_decode_attention_tree,
// pkv_prefill_attention_window): checks, choice of the kernel, and the merge of the states
// that the tree kernels leave where a unit of work was split.
#include <algorithm>
#include <type_traits>

#include "rows.cuh"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kCombineWarps = 8;

struct CombineParams {
  PlanParams plan;
  const float* part;
  char* out;
  int hq, D, f32, grid;  // grid: CTAs of a line of the kernel that left the states
  int lines;
  int blocks_seq;        // CTAs of a sequence
  int rows_warp;         // rows a warp takes, one after the other
  Repair repair;
};

// One (token, query head) row, by one warp: the states of its unit in the CTAs that shared it,
// by the log-sum-exp rule.  Rows that one CTA finished are left alone.
// kInFlight: states that a warp loads at once, where there are more than 4.
template <int kInFlight>
__device__ __forceinline__ void combine_row(const CombineParams& p, const SeqPlan& q, int b,
                                            long long chunk, long long before, int row) {
  const int lane = threadIdx.x & 31;
  const int tok = row / p.hq, h = row - tok * p.hq, g = h / p.plan.G;
  const int r = tok * p.plan.G + h - g * p.plan.G, ur = p.plan.unit_rows, unit = r / ur;
  const bool own_line = p.lines > 1;  // of the kv head
  const long long start =
      before + ((long long)(own_line ? 0 : g) * q.nru + unit) * q.steps + p.plan.lead;
  const long long c0 = div_pos(start, chunk), c1 = div_pos(start + q.t.nt - 1, chunk);
  if (c0 == c1) return;
  const long long row_floats = p.D + 4, slot = ur * row_floats, stride = 2 * p.lines * slot;
  const float* first = p.part + (r - unit * ur) * row_floats + c0 * stride +
                       (own_line ? 2 * g * slot : 0);
  const int pieces = (int)(c1 - c0) + 1, d = lane * 4;
  float top = -INFINITY, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
  // a state's numbers and values are loaded together: one round trip for N of them
  auto merge = [&](auto n, int i0) {
    constexpr int N = decltype(n)::value;
    float2 ml[N];
    float4 y[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      ml[u] = make_float2(-INFINITY, 0.f);
      y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + u < pieces) {
        // (the CTA with the unit's first tile left its part in its second slot)
        const float* s = first + (i0 + u) * stride + (i0 + u == 0 ? slot : 0);
        ml[u] = *reinterpret_cast<const float2*>(s);
        if (d < p.D) y[u] = *reinterpret_cast<const float4*>(s + 4 + d);
      }
    }
    float most = top;
#pragma unroll
    for (int u = 0; u < N; ++u) most = fmaxf(most, ml[u].x);
    const float shrink = most == top ? 1.f : exp2f(top - most);
    top = most;
    sum *= shrink;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= shrink;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      // a state at -inf saw nothing, or only NaN: its sum and O are 0, or NaN
      const float f = ml[u].x == -INFINITY ? 1.f : exp2f(ml[u].x - top);
      sum += f * ml[u].y;
      x[0] += f * y[u].x;
      x[1] += f * y[u].y;
      x[2] += f * y[u].z;
      x[3] += f * y[u].w;
    }
  };
  // (states that are not there cost as much as the others: 16 trees of 64 tokens, of 2 to 4 states a
  // row, 208 us with kInFlight alone, 203; two rows at once, for more loads in flight, took registers
  // that warps need more: 206)
  if (pieces <= 2) {
    merge(std::integral_constant<int, 2>(), 0);
  } else if (pieces <= 4) {
    merge(std::integral_constant<int, 4>(), 0);
  } else {
    for (int i0 = 0; i0 < pieces; i0 += kInFlight)
      merge(std::integral_constant<int, kInFlight>(), i0);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no weight at all: zeros
  const long long dst = ((q.s.q0 + tok) * p.hq + h) * p.D + d;
  if (d < p.D) {
    if (p.f32)
      *reinterpret_cast<float4*>(p.out + dst * 4) =
          make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    else
      *reinterpret_cast<uint2*>(p.out + dst * 2) =
          make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
  }
  // (lanes behind the dims hold zeros)
  const bool bad = nonfinite(x[0]) || nonfinite(x[1]) || nonfinite(x[2]) || nonfinite(x[3]);
  if (__any_sync(0xffffffffu, bad) && !nonfinite(sum)) repair_row<-1, 1>(p.repair, b, tok, h);
}

// A CTA takes kCombineWarps * rows_warp rows of one sequence.
template <int KT, int kInFlight>
__global__ void __launch_bounds__(kCombineWarps * 32)
    tree_combine_kernel(const __grid_constant__ CombineParams p) {
  __shared__ long long scratch[32];
  // What stands before the wait reads inputs alone, which were complete when the grid that
  // leaves the states let this one launch: it runs beside that grid's end.
  const int b = blockIdx.x / p.blocks_seq;
  const int first_row = (blockIdx.x - b * p.blocks_seq) * (kCombineWarps * p.rows_warp);
  const SeqPlan q = seq_plan<KT>(p.plan, b);
  if (first_row >= q.s.n * p.hq) {
    griddep_wait();
    griddep_launch_dependents();
    return;
  }
  const PlanSums sums = plan_sums<KT>(p.plan, b, scratch);
  const long long chunk = plan_chunk(sums.total, p.grid), before = sums.before;
  griddep_wait();
  griddep_launch_dependents();
  for (int i = 0; i < p.rows_warp; ++i) {
    const int row = first_row + i * kCombineWarps + (int)(threadIdx.x >> 5);
    if (row >= q.s.n * p.hq) break;
    combine_row<kInFlight>(p, q, b, chunk, before, row);
  }
}

// One CTA a sequence: its numbers, and the entries of the blocks that hold a seen key.
__global__ void validate_spans_kernel(const SpanParams p, const int32_t* q_pos,
                                      const unsigned long long* mask, int words, const int32_t* bt,
                                      long long num_blocks, int* err) {
  const int b = blockIdx.x;
  const SeqSpan s = seq_span(p, b);
  if (s.bad && threadIdx.x == 0) set_error(err, kErrCapacity);
  if (!s.ok) return;
  const int last = s.off + s.ctx + s.n - 1, lo = s.off + window_start(s.ctx, p.window);
  const int sink_end = min(s.off + p.sink, last + 1);
  for (int e = threadIdx.x; e <= last / p.bs; e += blockDim.x) {
    const int first = max(s.off, e * p.bs), end = min(last + 1, (e + 1) * p.bs);
    if (end <= lo && first >= sink_end) continue;
    const int blk = bt[(long long)b * p.mb + e];
    if (blk < 0 || blk >= num_blocks) report_entry(p, q_pos, mask, words, b, e, err);
  }
}

// Rows of a unit of the mma.sync kernels, where a sequence has up to `rows` of a kv head.
int rows_unit(const PoolView& v, int64_t rows) {
  const int most = v.io_size == 4 && v.head_dim == 128 ? 32 : 64;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : most;
}

// How a tree call runs: units of unit_rows rows, split over `grid` CTAs.  tcgen05, where it can,
// from more than 16 rows of a kv head on with head_dim 128, 32 with 64 (its work does not depend
// on the rows, that of mma.sync does).  mma.sync and tcgen05, 8 kv heads, groups of 4, D 128: 16
// rows, 16 sequences on 8192 91 and 101 us, one on 8192 18 and 20; 32 rows 103 and 103, one on
// 16384 27 and 25, on 30000 41 and 38; 64 rows 152 and 108.  D 64: 32 rows, 16 sequences on 8192
// 70 and 87, one on 30000 28 and 30; 64 rows 109 and 91.
struct TreePath {
  bool tcgen05;
  int unit_rows, grid;
  int lines;     // 1, or num_kv_heads: each kv head's units are a line of their own
  size_t bytes;  // of workspace
};

TreePath tree_path(const PoolView& v, int G, int max_q_len, int sms) {
  TreePath t;
  t.lines = 1;
  const long long rows = (long long)max_q_len * G;
  t.tcgen05 = rows > (v.head_dim == 128 ? 16 : 32) && span_supported(v, G * v.num_kv_heads, false);
  if (t.tcgen05) {
    const int tile = 128 / G * G;  // rows of whole tokens
    t.unit_rows = rows <= tile ? tile : 2 * tile;
    t.grid = sms;
    t.bytes = (size_t)2 * t.grid * t.unit_rows * (v.head_dim + 4) * 4;
    return t;
  }
  t.unit_rows = rows_unit(v, rows);
  const int ctas = v.quant          ? rows_ctas_i8(v.head_dim, t.unit_rows)
                   : v.io_size == 2 ? rows_ctas_bf16(v.head_dim, t.unit_rows)
                                    : rows_ctas_f32(v.head_dim, t.unit_rows);
  t.grid = sms * ctas;
  // int8: a row's codes of one head share their last lines with the next head's, and the scales of
  // all heads are one sector: where the heads are read at the same time, each comes from memory
  // once.  So each head's line is split in the same way, and CTAs of one place follow one another,
  // unless that leaves more than a tenth of the grid without work (32 trees of 4 to 8 tokens behind
  // 1024 to 8192: 579 MB and 125 us in one line, 327 MB and 122 us).
  if (v.quant) {
    const int pieces = t.grid / v.num_kv_heads;
    if (pieces > 0 && (t.grid - pieces * v.num_kv_heads) * 10 <= t.grid) {
      t.lines = v.num_kv_heads;
      t.grid = pieces * t.lines;
    }
  }
  t.bytes = (size_t)2 * t.grid * t.unit_rows * (v.head_dim + 4) * 4;
  return t;
}

cudaError_t launch_rows(const PoolView& v, const RowsParams& p, bool tree, long long grid, int dev,
                        cudaStream_t s) {
  if (v.quant) return launch_rows_i8(p, v.head_dim, tree, grid, dev, s);
  if (v.io_size == 2) return launch_rows_bf16(p, v.head_dim, tree, grid, dev, s);
  return launch_rows_f32(p, v.head_dim, tree, grid, dev, s);
}

// Whether a windowed prefill takes the tcgen05 kernel, where both could.  It works on whole
// windows of 4 tiles of 128 rows a CTA pair; the mma.sync kernel shares a unit's keys out over a
// cluster where units are few.  Estimated from a tile's time in us (128 keys x 2 tiles a CTA; 64
// keys x 64 rows a CTA, beside the others of its SM) and what an item costs besides.  On 4096
// under a window of 4096, 32 / 8 heads, D 128, tcgen05 and mma.sync took for 30 tokens 68 and 26
// us, 100 tokens 78 and 45, 300 tokens 79 and 80, 512 tokens 79 and 146; under a window of 500,
// 100 tokens 21 and 17, 512 tokens 21 and 30; with D 64, 100 tokens 69 and 34.  Over 448 shapes (1 to 16
// sequences of 16 to 4096 tokens behind windows of 128 to 8192, 4 and 8 kv heads, groups of 1 to 16, both D),
// each measured on both kernels, the one chosen was never more than 1.12 of the other, nor 7 us above it.
bool prefill_on_tcgen05(const PoolView& v, const RowsParams& p, int sms) {
  if (!span_supported(v, p.hq, true) || p.plan.unit_rows <= 32) return false;
  const bool d64 = v.head_dim == 64;
  const double heads = (double)p.plan.span.batch * v.num_kv_heads;
  const int tokens = 128 / p.plan.G, tiles_q = (p.plan.span.max_q_len + tokens - 1) / tokens;
  const double items = (tiles_q + 3) / 4 * heads;
  const double pairs_us =
      std::ceil(items / (sms / 2)) * (p.keys_most / 128. * (d64 ? 1.9 : 2.3) + 8);
  const double units = p.units_max * heads, held = sms * rows_ctas_bf16(v.head_dim, 64);
  int ctas = kRowsMaxCluster;
  while (ctas > 1 && units * ctas > held) ctas >>= 1;
  const double rows_us =
      std::ceil(units * ctas / held) * (p.keys_most / 64. / ctas * (d64 ? 1.6 : 2.3) + 7);
  return pairs_us <= rows_us;
}

// The arguments that the two calls share.
struct Call {
  const pkv_pool* pool;
  int32_t layer;
  const void* q;
  int32_t num_q_heads;
  float scale;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t *seq_lens, *offsets;
  const int64_t* cu_q;
  int32_t batch;
  int64_t total_q;
  int32_t max_q_len, window, sink;
  void* out;
};

// Their checks, in the order of the other calls.  *empty: there is nothing to compute.
int check_call(const Call& c, PoolView* v, bool* empty) {
  const int st = pool_view(c.pool, true, v);
  if (st != PKV_OK) return st;
  if (c.layer < 0 || c.layer >= v->num_layers || c.batch < 0 || c.num_q_heads <= 0 ||
      c.total_q < 0 || c.max_q_len < 0 || c.window < 0 || c.sink < 0 ||
      c.num_q_heads % v->num_kv_heads != 0 || !std::isfinite(c.scale))
    return PKV_ERR_INVALID_ARG;
  if ((v->head_dim != 64 && v->head_dim != 128) || c.num_q_heads / v->num_kv_heads > 16)
    return PKV_ERR_UNSUPPORTED;
  *empty = c.batch == 0 || c.total_q == 0 || c.max_q_len == 0;
  if (*empty) return PKV_OK;
  if (!c.q || !c.out || !c.block_tables || !c.seq_lens || !c.cu_q || c.max_blocks_per_seq <= 0)
    return PKV_ERR_INVALID_ARG;
  if (!aligned(c.q, 16) || !aligned(c.out, 16) || !aligned(c.block_tables, 4) ||
      !aligned(c.seq_lens, 4) || !aligned(c.offsets, 4) || !aligned(c.cu_q, 8))
    return PKV_ERR_INVALID_ARG;
  // rows, positions and grids are 32-bit in the kernels
  const int64_t units = ((int64_t)c.max_q_len * c.num_q_heads + 7) / 8;
  if ((int64_t)c.max_blocks_per_seq * v->block_size > kMaxPositions || c.total_q > INT32_MAX ||
      c.batch > 65535 || units * c.batch > INT32_MAX || units > (1 << 26))
    return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

RowsParams rows_params(const Call& c, const PoolView& v, int* err) {
  RowsParams p = {};
  SpanParams& s = p.plan.span;
  s.lens = c.seq_lens;
  s.offs = c.offsets;
  s.cu_q = reinterpret_cast<const long long*>(c.cu_q);
  s.total_q = c.total_q;
  s.batch = c.batch;
  s.mb = c.max_blocks_per_seq;
  s.bs = v.block_size;
  s.max_q_len = c.max_q_len;
  s.window = c.window;
  s.sink = c.sink < kMaxPositions ? c.sink : (int)kMaxPositions;
  s.gran = 1;
  p.plan.G = c.num_q_heads / v.num_kv_heads;
  p.plan.hkv = v.num_kv_heads;
  p.k = v.k;
  p.v = v.v;
  p.q = static_cast<const char*>(c.q);
  p.out = static_cast<char*>(c.out);
  p.bt = c.block_tables;
  p.err = err;
  p.num_blocks = v.num_blocks;
  p.L = v.num_layers;
  p.layer = c.layer;
  p.row_bytes = v.row_bytes;
  p.scale_off = v.scale_off;
  p.hq = c.num_q_heads;
  while (1 << p.bs_bits < v.block_size) ++p.bs_bits;
  p.qscale = c.scale * kLog2e;
  Repair& r = p.repair;
  r.span = s;
  r.k = v.k;
  r.v = v.v;
  r.q = p.q;
  r.out = p.out;
  r.bt = p.bt;
  r.num_blocks = v.num_blocks;
  r.hq = c.num_q_heads;
  r.G = p.plan.G;
  r.L = v.num_layers;
  r.layer = c.layer;
  r.bs_bits = p.bs_bits;
  r.row_bytes = v.row_bytes;
  r.scale_off = v.scale_off;
  r.D = v.head_dim;
  r.dtype = c.pool->dtype;
  r.qscale = p.qscale;
  return p;
}

int validate_call(const RowsParams& p, cudaStream_t stream) {
  int st;
  if ((st = clear_error_word(p.err, stream)) != PKV_OK) return st;
  if ((st = launch_status(launch_validate_spans(p.plan.span, p.q_pos, p.mask, p.words, p.bt,
                                                p.num_blocks, p.err, stream))) != PKV_OK)
    return st;
  return read_and_clear_error_word(p.err, stream);
}

}  // namespace

cudaError_t launch_validate_spans(const SpanParams& p, const int32_t* q_pos,
                                  const unsigned long long* mask, int words, const int32_t* bt,
                                  long long num_blocks, int* err, cudaStream_t s) {
  validate_spans_kernel<<<(unsigned)p.batch, 128, 0, s>>>(p, q_pos, mask, words, bt, num_blocks, err);
  return cudaGetLastError();
}

}  // namespace pkv

extern "C" {

size_t pkv_decode_tree_workspace_size(const pkv_pool* pool, int32_t batch, int32_t num_q_heads,
                                      int32_t max_q_len) {
  pkv::PoolView v;
  if (pkv::pool_view(pool, false, &v) != PKV_OK) return 0;
  if (batch < 0 || num_q_heads <= 0 || num_q_heads % v.num_kv_heads != 0 || max_q_len < 0) return 0;
  if (v.head_dim != 64 && v.head_dim != 128) return 0;
  int sms;
  if (pkv::device_sm_count(&sms) != PKV_OK) return 0;
  return pkv::tree_path(v, num_q_heads / v.num_kv_heads, max_q_len, sms).bytes;
}

pkv_status pkv_decode_attention_tree(const pkv_pool* pool, int32_t layer, const void* q,
                                     int32_t num_q_heads, float scale, const int32_t* block_tables,
                                     int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                     const int32_t* offsets, const int64_t* cu_q, int32_t batch,
                                     int64_t total_q, int32_t max_q_len, const uint64_t* tree_mask,
                                     int32_t mask_words, const int32_t* q_pos, int32_t window,
                                     int32_t sink, void* out, void* workspace,
                                     size_t workspace_bytes, cudaStream_t stream) {
  const pkv::Call c = {pool, layer, q, num_q_heads, scale, block_tables, max_blocks_per_seq,
                       seq_lens, offsets, cu_q, batch, total_q, max_q_len, window, sink, out};
  pkv::PoolView v;
  bool empty;
  int st = pkv::check_call(c, &v, &empty);
  if (st != PKV_OK) return (pkv_status)st;
  // the mask has a bit for each drafted token; positions go with a mask
  if (tree_mask ? mask_words < 1 || max_q_len > (int64_t)64 * mask_words
                : mask_words != 0 || q_pos != nullptr)
    return PKV_ERR_INVALID_ARG;
  if (empty) return PKV_OK;
  if (!pkv::aligned(tree_mask, 8) || !pkv::aligned(q_pos, 4)) return PKV_ERR_INVALID_ARG;
  if (!workspace || !pkv::aligned(workspace, 16)) return PKV_ERR_WORKSPACE;
  int optin, decode_grid, validate, sms, dev;
  int* err;
  if ((st = pkv::device_facts(&optin, &err, &decode_grid, &validate)) != PKV_OK)
    return (pkv_status)st;
  if ((st = pkv::device_sm_count(&sms, &dev)) != PKV_OK) return (pkv_status)st;
  pkv::RowsParams p = pkv::rows_params(c, v, err);
  const pkv::TreePath path = pkv::tree_path(v, p.plan.G, max_q_len, sms);
  if (workspace_bytes < path.bytes) return PKV_ERR_WORKSPACE;
  p.plan.unit_rows = path.unit_rows;
  p.plan.lead = path.tcgen05 ? 2 : 4;
  p.lines = path.lines;
  if (path.lines > 1) p.plan.hkv = 1;
  if (path.tcgen05) p.plan.span.gran = v.block_size;  // (tensor copies of whole blocks)
  p.part = static_cast<float*>(workspace);
  p.mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  p.words = mask_words;
  p.q_pos = q_pos;
  p.repair.mask = p.mask;
  p.repair.words = mask_words;
  p.repair.q_pos = q_pos;
  if (validate && (st = pkv::validate_call(p, stream)) != PKV_OK) return (pkv_status)st;
  const cudaError_t e =
      path.tcgen05
          ? pkv::launch_prefill_tree(v, layer, q, num_q_heads, scale, block_tables, p.plan, q_pos,
                                     p.mask, mask_words, p.repair, p.part, out, err, sms, stream)
          : pkv::launch_rows(v, p, true, path.grid, dev, stream);
  if ((st = pkv::launch_status(e)) != PKV_OK) return (pkv_status)st;
  pkv::CombineParams m = {};
  m.plan = p.plan;
  m.part = p.part;
  m.out = p.out;
  m.hq = num_q_heads;
  m.D = v.head_dim;
  m.f32 = v.io_size == 4;
  m.grid = path.grid / path.lines;
  m.lines = path.lines;
  m.repair = p.repair;
  // as many CTAs as the device holds about at once: each goes over the batch first
  const int64_t rows = (int64_t)max_q_len * num_q_heads;
  const int64_t all = rows * batch / pkv::kCombineWarps;
  m.rows_warp = (int)std::max<int64_t>(1, std::min<int64_t>(64, all / (6 * sms)));
  const int64_t cta_rows = (int64_t)pkv::kCombineWarps * m.rows_warp;
  m.blocks_seq = (int)((rows + cta_rows - 1) / cta_rows);
  const int keys = path.tcgen05 ? 128 : pkv::rows_tile_keys(pool->dtype, path.unit_rows);
  // Few CTAs: a long context's states are a chain of loads, 16 at a time (one tree of 24 tokens on
  // 16384 28.0 us with 8, 26.4; of 8 on 30000 44.1, 41.0).  Many: registers for more of them (16
  // trees of 64 tokens 206 us with 8, 220 with 16).
  const bool few = (int64_t)m.blocks_seq * batch <= 2 * sms;
  const auto kern =
      few ? keys == 128  ? pkv::tree_combine_kernel<128, 16>
            : keys == 64 ? pkv::tree_combine_kernel<64, 16>
                         : pkv::tree_combine_kernel<32, 16>
          : keys == 128  ? pkv::tree_combine_kernel<128, 8>
            : keys == 64 ? pkv::tree_combine_kernel<64, 8>
                         : pkv::tree_combine_kernel<32, 8>;
  st = pkv::launch_status(pkv::launch_kernel(kern, dim3((unsigned)(m.blocks_seq * batch)),
                                             dim3(pkv::kCombineWarps * 32), 0, stream, true, m));
  if (st != PKV_OK) return (pkv_status)st;
  return validate ? (pkv_status)pkv::read_and_clear_error_word(err, stream) : PKV_OK;
}

pkv_status pkv_prefill_attention_window(const pkv_pool* pool, int32_t layer, const void* q,
                                        int32_t num_q_heads, float scale,
                                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                                        const int32_t* seq_lens, const int32_t* offsets,
                                        const int64_t* cu_q, int32_t batch, int64_t total_q,
                                        int32_t max_q_len, int32_t window, int32_t sink, void* out,
                                        cudaStream_t stream) {
  const pkv::Call c = {pool, layer, q, num_q_heads, scale, block_tables, max_blocks_per_seq,
                       seq_lens, offsets, cu_q, batch, total_q, max_q_len, window, sink, out};
  pkv::PoolView v;
  bool empty;
  int st = pkv::check_call(c, &v, &empty);
  if (st != PKV_OK) return (pkv_status)st;
  if (window < 1) return PKV_ERR_INVALID_ARG;
  if (empty) return PKV_OK;
  int optin, decode_grid, validate, sms, dev;
  int* err;
  if ((st = pkv::device_facts(&optin, &err, &decode_grid, &validate)) != PKV_OK)
    return (pkv_status)st;
  if ((st = pkv::device_sm_count(&sms, &dev)) != PKV_OK) return (pkv_status)st;
  pkv::RowsParams p = pkv::rows_params(c, v, err);
  const int64_t rows = (int64_t)max_q_len * p.plan.G;
  p.plan.unit_rows = pkv::rows_unit(v, rows);
  if (validate && (st = pkv::validate_call(p, stream)) != PKV_OK) return (pkv_status)st;
  p.units_max = (int)((rows + p.plan.unit_rows - 1) / p.plan.unit_rows);
  const int64_t held = (int64_t)max_blocks_per_seq * v.block_size;
  p.keys_most = std::min(held, (int64_t)window + p.plan.span.sink + p.plan.unit_rows / p.plan.G);
  const int asked = pkv::debug_window_path();
  if (asked == 2 && !pkv::span_supported(v, num_q_heads, true)) return PKV_ERR_UNSUPPORTED;
  const cudaError_t e =
      (asked == 0 ? pkv::prefill_on_tcgen05(v, p, sms) : asked == 2)
          ? pkv::launch_prefill(v, layer, q, num_q_heads, scale, block_tables, max_blocks_per_seq,
                                seq_lens, offsets, cu_q, batch, total_q, max_q_len, window,
                                p.plan.span.sink, out, err, sms, stream, &p.repair)
          : pkv::launch_rows(v, p, false, 0, dev, stream);
  if ((st = pkv::launch_status(e)) != PKV_OK) return (pkv_status)st;
  return validate ? (pkv_status)pkv::read_and_clear_error_word(err, stream) : PKV_OK;
}

}  // extern "C"
