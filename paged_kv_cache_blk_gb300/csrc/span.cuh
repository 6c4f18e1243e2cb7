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

// ---- one list of tiles for a batch, split evenly over a grid --------------------------
//
// A unit is UR query rows (tokens x heads of a group) of one sequence and kv head over
// all of the sequence's tiles.  The units of all sequences in order, tile by tile, are
// one line of T tiles; CTA c takes the tiles [c * chunk, (c + 1) * chunk) of it, so
// every CTA has the same work whatever the lengths.  A unit that lies in one CTA's share
// is finished there; of the others each CTA leaves the state of its part in slot
// 2 c (a unit that began before the share) or 2 c + 1 (one that goes on behind it), and a
// second kernel merges them.

struct PlanParams {
  SpanParams span;
  int unit_rows;  // UR
  int G, hkv;
  int least;  // tiles of a share at least
};

struct SeqPlan {
  SeqSpan s;
  KeyList t;
  int nru;  // units of one kv head
  long long tiles;
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
  q.tiles = (long long)q.t.nt * q.nru * p.hkv;
  return q;
}

// a / b for positive numbers, by the short division where they fit.
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

__device__ __forceinline__ long long plan_chunk(const PlanParams& p, long long total, int grid) {
  const long long c = div_pos(total + grid - 1, grid);
  return c > p.least ? c : p.least;
}

// What the merge needs of the line: its length, and the tiles before one sequence.
struct PlanSums {
  long long total, before;
};

// A CTA's share: tiles at .. end - 1, the first of them in sequence b, whose own tiles begin
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
    const long long tiles = seq_plan<KT>(p, b).tiles;
    all += tiles;
    before += b < seq ? tiles : 0;
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
  long long mine = tid < p.span.batch ? seq_plan<KT>(p, tid).tiles : 0;
  long long total, incl = block_scan(mine, s, &total);
  for (int b0 = n; b0 < p.span.batch; b0 += n) {
    long long all;
    block_scan(b0 + tid < p.span.batch ? seq_plan<KT>(p, b0 + tid).tiles : 0, s, &all);
    total += all;
  }
  const long long chunk = plan_chunk(p, total, grid);
  const long long at = min(total, cta * chunk), end = min(total, at + chunk);
  if (at >= end) return PlanShare{at, end, 0, 0};
  long long base = 0;
  for (int b0 = 0;; b0 += n) {
    long long all = total;
    if (!once) {
      mine = b0 + tid < p.span.batch ? seq_plan<KT>(p, b0 + tid).tiles : 0;
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
// seen, for validate mode.
cudaError_t launch_validate_spans(const SpanParams& p, const int32_t* bt, long long num_blocks,
                                  int* err, cudaStream_t s);

// Host side (prefill.cu, where prefill_supported): the tree decode on tcgen05, units of 256
// rows, or of 128 where none has more, key tiles of 128, split over a grid of sm_count CTAs.
cudaError_t launch_prefill_tree(const PoolView& pv, int layer, const void* q, int num_q_heads,
                                float scale, const int32_t* bt, const PlanParams& plan,
                                const int32_t* q_pos, const unsigned long long* mask, int words,
                                float* part, void* out, int* err, int sm_count, cudaStream_t s);

}  // namespace pkv
