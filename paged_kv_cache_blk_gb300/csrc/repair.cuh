// Results that a value which their query does not see has spoiled.
//
// The kernels multiply a tile's V rows by the weights of several queries at once, 0 where a
// query does not see a row; 0 times an infinity or a NaN is NaN.  A result that came out NaN or
// infinite although its weights' sum is finite (scores of seen keys decide that sum alone) is
// computed again over the seen keys only, a warp a row: lanes over the dims, each score once.
//
// Where: nothing waits for it.  prefill.cu marks such rows and goes on; a CTA computes its marked
// rows after its last item, when its pipeline is over and its tensor memory free, so that however
// long a context they have, no bounded wait of the launch runs out on them.  The mma.sync kernels
// do it between pieces and tree_combine_kernel after a row; neither has such waits.  Off the usual
// path: no speed is sought beyond that, and the call takes few values so that the kernels keep
// theirs in registers.
#pragma once

#include "common.cuh"
#include "span.cuh"

namespace pkv {

__device__ __forceinline__ bool nonfinite(float x) { return (__float_as_uint(x) << 1) >= 0xff000000u; }

// A bf16 NaN that no conversion gives: the first element of (a half of) a row that is to be
// computed again.
constexpr unsigned short kSpoiled = 0x7fd5;

struct Repair {
  SpanParams span;
  const char* k;
  const char* v;
  const char* q;
  char* out;
  const int32_t* bt;
  const int32_t* q_pos;            // as in RowsParams
  const unsigned long long* mask;
  long long num_blocks;
  int words, hq, G, L, layer, bs_bits, row_bytes, scale_off, D, dtype;  // dtype: of the pool
  float qscale;  // scale * log2(e)
};

// E elements of a row from number i on (a multiple of E), E = 2 or 4.
template <int E>
__device__ __forceinline__ void repair_elements(const char* row, int dtype, int i, float (&x)[E]) {
  if (dtype == PKV_F32) {
    const float2* a = reinterpret_cast<const float2*>(row) + i / 2;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) x[2 * e] = a[e].x, x[2 * e + 1] = a[e].y;
  } else if (dtype == PKV_BF16) {
    const uint32_t* a = reinterpret_cast<const uint32_t*>(row) + i / 2;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) x[2 * e] = bf16_lo(a[e]), x[2 * e + 1] = bf16_hi(a[e]);
  } else {
    const uchar2* a = reinterpret_cast<const uchar2*>(row) + i / 2;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) x[2 * e] = a[e].x - 128.f, x[2 * e + 1] = a[e].y - 128.f;
  }
}

// The result of token tok and query head h of sequence b.
template <int E>
static __device__ __noinline__ void repair_row_of(const Repair& p, int b, int tok, int h) {
  constexpr unsigned kWarp = 0xffffffffu;
  constexpr int kKeysAtOnce = 4;
  const int lane = threadIdx.x & 31, d = lane * E;
  const SeqSpan s = seq_span(p.span, b);
  const int last = p.mask ? s.ctx + s.n - 1 : s.ctx + tok, g = h / p.G, first = g * p.D + d;
  const KeyList t = key_list<32>(p.span, s.off, window_start(s.ctx, p.span.window), last);
  const long long query = s.q0 + tok, at_q = (query * p.hq + h) * p.D;
  const RowSees sees = row_sees(p.span, t, s.off, s.ctx, s.n, tok, query, p.q_pos, p.mask, p.words);
  const int io = p.dtype == PKV_F32 ? PKV_F32 : PKV_BF16;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  repair_elements<E>(p.q + at_q * (io == PKV_F32 ? 4 : 2), io, d, q);
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int x0 = 0; x0 < t.nt * 32; x0 += 32) {
    uint32_t todo = sees.bits_from(x0);  // the same in every lane
    // each lane looks up the row of one place; -1: a block outside the pool, which reads as zeros
    long long at = -1;
    if (todo >> lane & 1) {
      const int pos = t.position(x0 + lane);
      const int blk = p.bt[(long long)b * p.span.mb + (pos >> p.bs_bits)];
      if (blk >= 0 && blk < p.num_blocks)
        at = ((((long long)blk * p.L + p.layer) << p.bs_bits) + (pos & ((1 << p.bs_bits) - 1))) *
             p.row_bytes;
    }
    while (todo) {
      float x[kKeysAtOnce], v[kKeysAtOnce][E];
      bool on[kKeysAtOnce];
      float top = m;
#pragma unroll
      for (int u = 0; u < kKeysAtOnce; ++u) {
        on[u] = todo != 0;
        const int key = on[u] ? __ffs(todo) - 1 : 0;
        todo &= todo - 1;
        const long long row = __shfl_sync(kWarp, at, key);
        x[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] = 0.f;
        if (on[u] && row >= 0) {
          float k[E];
          repair_elements<E>(p.k + row, p.dtype, first, k);
          repair_elements<E>(p.v + row, p.dtype, first, v[u]);
#pragma unroll
          for (int e = 0; e < E; ++e) x[u] = fmaf(q[e], k[e], x[u]);
          if (p.dtype == PKV_I8) {
            x[u] *= *reinterpret_cast<const float*>(p.k + row + p.scale_off + 4 * g);
            const float sv = *reinterpret_cast<const float*>(p.v + row + p.scale_off + 4 * g);
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] *= sv;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kKeysAtOnce; ++u) {
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) x[u] += __shfl_xor_sync(kWarp, x[u], i);
        x[u] = on[u] ? x[u] * p.qscale : -INFINITY;
        top = fmaxf(top, x[u]);
      }
      const float shrink = m == -INFINITY ? 0.f : exp2f(m - top);
      m = top;
      l *= shrink;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= shrink;
#pragma unroll
      for (int u = 0; u < kKeysAtOnce; ++u) {
        const float w = x[u] == -INFINITY ? 0.f : exp2f(x[u] - top);
        l += w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, v[u][e], o[e]);
      }
    }
    // a NaN in every dim stays
    bool lost = true;
#pragma unroll
    for (int e = 0; e < E; ++e) lost &= o[e] != o[e];
    if (__all_sync(kWarp, lost)) break;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const long long i = at_q + d + e;
    if (io == PKV_F32)
      *reinterpret_cast<float2*>(p.out + i * 4) = make_float2(o[e] * inv, o[e + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(p.out + i * 2) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  }
}

// By a whole warp; what its lanes stored of the row before is replaced.
__device__ __forceinline__ void repair_row(const Repair& p, int b, int tok, int h) {
  __syncwarp();
  if (p.D == 64)
    repair_row_of<2>(p, b, tok, h);
  else
    repair_row_of<4>(p, b, tok, h);
}

}  // namespace pkv
