// Which keys the new tokens of a sequence see under a window, first tokens that
// stay visible and a mask among the new tokens (rows.cuh, prefill.cu), the key
// tiles that hold them, and how the tiles of a batch are split over a grid.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace pkv {

// Host limit on max_blocks_per_seq * block_size: table positions, and sums of two
// of them, are 32-bit in the kernels.
constexpr long long kMaxPositions = 1ll << 30;

struct SpanParams {
  const int32_t* lens;
  const int32_t* offs;
  const long long* cu_q;  // NULL: one new token a sequence
  long long total_q;
  int batch, mb, bs, max_q_len;
  int window;  // 0: none
  int sink;    // at most kMaxPositions
  int gran;    // lists of keys begin at multiples of it (a power of two, up to a key tile)
};

// The new tokens of sequence b: query rows q0 .. q0 + n - 1, its last n positions.
struct SeqSpan {
  long long q0;
  int n, ctx, off;
  bool ok;  // false: nothing is computed (bad: an error, and not just no tokens)
  bool bad;
};

__device__ __forceinline__ SeqSpan seq_span(const SpanParams& p, int b) {
  SeqSpan s;
  long long q1;
  if (p.cu_q) {
    s.q0 = p.cu_q[b];
    q1 = p.cu_q[b + 1];
  } else {
    s.q0 = b;
    q1 = b + 1;
  }
  const int len = p.lens[b];
  s.off = p.offs ? p.offs[b] : 0;
  const long long n = p.cu_q || len != 0 ? q1 - s.q0 : 0;
  s.bad = n < 0 || (n > 0 && (n > p.max_q_len || s.q0 < 0 || q1 > p.total_q || len < n || s.off < 0 ||
                    s.off >= p.bs || (long long)s.off + len > (long long)p.mb * p.bs));
  s.ok = n > 0 && !s.bad;
  s.n = s.ok ? (int)n : 0;
  s.ctx = len - s.n;
  return s;
}

// The keys that some of the queries see, in a row: the first tokens, then those from the
// earliest window on, each from and up to a multiple of `gran` table positions.  Place x of
// the list holds table position x + s0 where x < head, x + shift behind; tile i is places
// i KT .. i KT + KT - 1, nt tiles in all.  (Where the two parts meet, s0 = shift.)
struct KeyList {
  int s0, head, shift, nt;
  __device__ __forceinline__ int position(int x) const { return x + (x < head ? s0 : shift); }
  // places of table positions: of one among the first tokens, of one from the windows on, and
  // of the last one that a row sees (which may lie before every window)
  __device__ __forceinline__ int first(int pos) const { return pos - (head > 0 ? s0 : shift); }
  __device__ __forceinline__ int behind(int pos) const { return pos - shift; }
  __device__ __forceinline__ int last(int pos) const {
    return pos - shift >= head ? pos - shift : min(pos - s0, head - 1);
  }
};

// lo: the key that the earliest window begins with; hi: the last key.
template <int KT>
__device__ __forceinline__ KeyList key_list(const SpanParams& p, int off, int lo, int hi) {
  KeyList t;
  const int down = -p.gran, w0 = (off + lo) & down;
  const int s = min(p.sink, lo);  // first tokens before the windows
  t.s0 = off & down;
  t.head = s > 0 ? max(0, min((off + s + p.gran - 1) & down, w0) - t.s0) : 0;
  t.shift = w0 - t.head;
  t.nt = (off + hi - t.shift + KT) / KT;
  return t;
}

// First key of the window of a query at position pos.
__device__ __forceinline__ int window_start(int pos, int window) {
  return window > 0 ? max(0, pos - window + 1) : 0;
}

// Places a .. b of the 32 from c0 on, as bits.
__device__ __forceinline__ uint32_t column_bits(int a, int b, int c0) {
  const int lo = max(a - c0, 0), hi = min(b - c0, 31);
  return lo > hi ? 0u : (0xffffffffu << lo) & (0xffffffffu >> (31 - hi));
}

// 32 drafted tokens from number d on (which may lie before the first) of a row's mask of n.
__device__ __forceinline__ uint32_t draft_bits(const unsigned long long* bits, int d, int n) {
  if (d <= -32 || d >= n) return 0;
  unsigned long long x;
  if (d < 0) {
    x = bits[0] << -d;
  } else {
    x = bits[d >> 6] >> (d & 63);
    // (the next word where the 32 go on in it and it holds drafted tokens)
    if ((d & 63) > 32 && ((d >> 6) + 1) * 64 < n) x |= bits[(d >> 6) + 1] << (64 - (d & 63));
  }
  return (uint32_t)x & column_bits(0, n - 1, d);
}

// What a query sees of a list: the places first .. top that are first tokens (before sink) or
// in its window (lo or later), and the drafted tokens, from place draft on, by their bits.
struct RowSees {
  int first, sink, lo, top, draft, n;
  const unsigned long long* bits;
  __device__ __forceinline__ bool all(int x, int keys) const {  // of places x .. x + keys - 1
    return x >= first && x + keys - 1 <= top && (x >= lo || x + keys <= sink);
  }
  __device__ __forceinline__ uint32_t bits_from(int x) const {  // of the 32 places from x on
    uint32_t w = column_bits(first, min(top, sink - 1), x) | column_bits(max(first, lo), top, x);
    if (bits) w |= draft_bits(bits, x - draft, n);
    return w;
  }
};

// Token tok of n new ones, query row `query` of the batch; q_pos and mask may be NULL (see
// pkv_decode_attention_tree).
__device__ __forceinline__ RowSees row_sees(const SpanParams& p, const KeyList& t, int off, int ctx,
                                            int n, int tok, long long query, const int32_t* q_pos,
                                            const unsigned long long* mask, int words) {
  RowSees r;
  r.first = t.first(off);
  r.sink = t.first(off + p.sink);
  r.top = t.last(off + (mask ? ctx - 1 : ctx + tok));
  r.draft = t.behind(off + ctx);
  r.n = n;
  r.bits = mask ? mask + query * words : nullptr;
  long long start = 0;
  if (p.window > 0) {
    const int pos = q_pos ? max(ctx, q_pos[query]) : ctx + tok;
    start = max(0ll, min((long long)pos - p.window + 1, kMaxPositions));
  }
  r.lo = t.behind(off + (int)start);
  return r;
}

// An entry of sequence b's table that is outside the pool: an error where some query sees a key of
// its block.  A windowed call lists no others; a tree's list begins with the window of a token right
// behind the context and holds every drafted token, so here the queries are asked (positions may all
// be later, and a bit may be set in no row).  Off the usual path.
static __device__ __noinline__ void report_entry(const SpanParams& p, const int32_t* q_pos,
                                                 const unsigned long long* mask, int words, int b,
                                                 int entry, int* err) {
  const SeqSpan s = seq_span(p, b);
  const int first = max(0, entry * p.bs - s.off);  // the block's keys: first .. end - 1
  const int end = min(s.ctx + s.n, (entry + 1) * p.bs - s.off);
  bool seen = mask == nullptr || (first < s.ctx && (p.window == 0 || first < p.sink));
  const int last_ctx = min(end, s.ctx) - 1, d0 = max(first, s.ctx) - s.ctx, d1 = end - 1 - s.ctx;
  for (int i = 0; i < s.n && !seen; ++i) {
    const long long query = s.q0 + i;
    const int pos = q_pos ? max(s.ctx, q_pos[query]) : s.ctx + i;
    seen = last_ctx >= first && last_ctx > (long long)pos - p.window;
    for (int w = d0 >> 6; d1 >= d0 && w <= d1 >> 6; ++w) {
      const int lo = max(d0 - 64 * w, 0), hi = min(d1 - 64 * w, 63);
      const unsigned long long of_block = (~0ull << lo) & (~0ull >> (63 - hi));
      seen |= (mask[query * words + w] & of_block) != 0;
    }
  }
  if (seen) set_error(err, kErrIndex);
}

// ---- one list of tiles for a batch, split evenly over a grid --------------------------
//
// A unit is UR query rows (tokens x heads of a group) of one sequence and kv head over
// all of the sequence's tiles, with `lead` steps of no work before them that stand for what a
// unit costs besides its tiles.  The units of all sequences in order, step by step, are one
// line of T steps; CTA c takes the steps [c * chunk, (c + 1) * chunk) of it, so every CTA has
// the same work whatever the lengths.  A unit whose tiles lie in one CTA's share is finished
// there; of the others each CTA leaves the state of its part in slot 2 c (a part that does not
// begin with the unit's first tile) or 2 c + 1, and a second kernel merges them.

struct PlanParams {
  SpanParams span;
  int unit_rows;  // UR
  int G, hkv;
  int lead;  // steps before a unit's tiles
};

struct SeqPlan {
  SeqSpan s;
  KeyList t;
  int nru;  // units of one kv head
  int steps;  // of a unit
  long long all_steps;
};

// A part of a unit: steps x .. of it, at most `most` of them.
struct PlanPart {
  int unit, t0, t1, steps;  // unit of the sequence (kv head major); tiles t0 .. t1 - 1
};


template <int KT>
__device__ __forceinline__ SeqPlan seq_plan(const PlanParams& p, int b) {
  SeqPlan q;
  q.s = seq_span(p.span, b);
  q.t = KeyList{0, 0, 0, 0};
  q.nru = 0;
  if (q.s.ok) {
    q.t = key_list<KT>(p.span, q.s.off, window_start(q.s.ctx, p.span.window),
                       q.s.ctx + q.s.n - 1);
    q.nru = (q.s.n * p.G + p.unit_rows - 1) / p.unit_rows;
  }
  q.steps = q.t.nt + p.lead;
  q.all_steps = (long long)q.steps * q.nru * p.hkv;
  return q;
}

// a / b for positive numbers, by the short division where they fit.
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// Steps of a share.
__device__ __forceinline__ long long plan_chunk(long long total, int grid) {
  return max(1ll, div_pos(total + grid - 1, grid));
}

// The part that begins `at` steps into the sequence's, up to `most` steps.
__device__ __forceinline__ PlanPart plan_part(const PlanParams& p, const SeqPlan& q, long long at,
                                              long long most) {
  PlanPart r;
  r.unit = (int)div_pos(at, q.steps);
  const int x = (int)(at - (long long)r.unit * q.steps);
  r.steps = (int)min((long long)(q.steps - x), most);
  r.t0 = max(0, x - p.lead);
  r.t1 = max(0, x + r.steps - p.lead);
  return r;
}

// What the merge needs of the line: its length, and the steps before one sequence.
struct PlanSums {
  long long total, before;
};

// A CTA's share: steps at .. end - 1, the first of them in sequence b, whose own steps begin
// at `first`.
struct PlanShare {
  long long at, end, first;
  int b;
};

// Inclusive sum of x over the threads of the block, and the sum over all (s: 32 words of shared
// memory).
__device__ __forceinline__ long long block_scan(long long x, long long* s, long long* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s[warp] = x;
  __syncthreads();
  long long sum = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    if (w < warp) x += s[w];
    sum += s[w];
  }
  *all = sum;
  return x;
}

// Over the whole block, which looks at each sequence once.
template <int KT>
__device__ __forceinline__ PlanSums plan_sums(const PlanParams& p, int seq, long long* s) {
  long long all = 0, before = 0;
  for (int b = threadIdx.x; b < p.span.batch; b += blockDim.x) {
    const long long steps = seq_plan<KT>(p, b).all_steps;
    all += steps;
    before += b < seq ? steps : 0;
  }
  PlanSums r;
  block_scan(all, s, &r.total);
  block_scan(before, s, &r.before);
  return r;
}

// Over the whole block.  Batches of up to blockDim.x sequences take one look at each.
template <int KT>
__device__ __forceinline__ PlanShare plan_share(const PlanParams& p, int cta, int grid,
                                                long long* s) {
  __shared__ PlanShare found;
  const int n = (int)blockDim.x, tid = threadIdx.x;
  const bool once = p.span.batch <= n;
  long long mine = tid < p.span.batch ? seq_plan<KT>(p, tid).all_steps : 0;
  long long total, incl = block_scan(mine, s, &total);
  for (int b0 = n; b0 < p.span.batch; b0 += n) {
    long long all;
    block_scan(b0 + tid < p.span.batch ? seq_plan<KT>(p, b0 + tid).all_steps : 0, s, &all);
    total += all;
  }
  const long long chunk = plan_chunk(total, grid);
  const long long at = min(total, cta * chunk), end = min(total, at + chunk);
  if (at >= end) return PlanShare{at, end, 0, 0};
  long long base = 0;
  for (int b0 = 0;; b0 += n) {
    long long all = total;
    if (!once) {
      mine = b0 + tid < p.span.batch ? seq_plan<KT>(p, b0 + tid).all_steps : 0;
      incl = block_scan(mine, s, &all);
    }
    const long long stop = base + incl;
    if (at >= stop - mine && at < stop) found = PlanShare{at, end, stop - mine, b0 + tid};
    base += all;
    if (at < base) break;
  }
  __syncthreads();
  return found;
}

// Host side (tree.cu): checks the sequences and the table entries that hold a key which is
// seen, for validate mode (trees: with their positions and mask).
cudaError_t launch_validate_spans(const SpanParams& p, const int32_t* q_pos,
                                  const unsigned long long* mask, int words, const int32_t* bt,
                                  long long num_blocks, int* err, cudaStream_t s);

struct Repair;  // repair.cuh

// Host side (prefill.cu): whether the tcgen05 kernels take a windowed prefill (pairs) or a tree.
bool span_supported(const PoolView& pv, int num_q_heads, bool pairs);
// The tree decode on them: units of two tiles of 128 / G tokens, or of one where no sequence has
// more; key tiles of 128; split over a grid of sm_count CTAs.
cudaError_t launch_prefill_tree(const PoolView& pv, int layer, const void* q, int num_q_heads,
                                float scale, const int32_t* bt, const PlanParams& plan,
                                const int32_t* q_pos, const unsigned long long* mask, int words,
                                const Repair& repair, float* part, void* out, int* err, int sm_count,
                                cudaStream_t s);

}  // namespace pkv
