// Results that a value which their query does not see has spoiled.
//
// The kernels multiply a tile's V rows by the weights of several queries at once, 0 where a
// query does not see a row; 0 times an infinity or a NaN is NaN.  A result that came out NaN or
// infinite although its weights' sum is finite (scores of seen keys decide that sum alone) is
// computed again over the seen keys only, a warp a row: lanes over the dims, each score once.  (Where
// the row does see it the result stays what it was.)
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

// Four elements of a row from number i on (a multiple of four).
__device__ __forceinline__ void repair_elements(const char* row, int dtype, int i, float (&x)[4]) {
  if (dtype == PKV_F32) {
    const float4 a = *reinterpret_cast<const float4*>(row + 4 * i);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  } else if (dtype == PKV_BF16) {
    const uint2 a = *reinterpret_cast<const uint2*>(row + 2 * i);
    x[0] = bf16_lo(a.x), x[1] = bf16_hi(a.x), x[2] = bf16_lo(a.y), x[3] = bf16_hi(a.y);
  } else {
    const uchar4 a = *reinterpret_cast<const uchar4*>(row + i);
    x[0] = a.x - 128.f, x[1] = a.y - 128.f, x[2] = a.z - 128.f, x[3] = a.w - 128.f;
  }
}

// The result of token tok and query head h of sequence b, by a whole warp, four dims a lane
// (head_dim 64: by half of it); what the lanes stored of the row before is replaced.
// kType: of the pool, or -1: p.dtype.  kKeysAtOnce: 4, whose loads are under way together, or 1 where
// the kernel pays for the registers of a call that it hardly ever makes (with 4 and 1, the call of one
// tree of 24 tokens on 16384 31.8 and 28.6 us, without repair in the merge 28.4; rows_tree_kernel, 32
// int8 trees, 121.8 and 118.4).  At worst, an infinity that all queries see, every row is computed
// again: 4096 tokens under a window of 1024, 32 / 8 heads, D 128, 14 ms on the tcgen05 kernel (39 with a
// third of the warps, 89 with branches between the loads too), 17 on the mma.sync one; NaN 0.7 and 0.5.
template <int kType, int kKeysAtOnce>
static __device__ __noinline__ void repair_row(const Repair& p, int b, int tok, int h) {
  constexpr unsigned kWarp = 0xffffffffu;
  constexpr int E = 4;
  __syncwarp();
  const int dtype = kType >= 0 ? kType : p.dtype;
  const int lane = threadIdx.x & 31, d = lane * E;
  const bool mine = d < p.D;
  const SeqSpan s = seq_span(p.span, b);
  const int last = p.mask ? s.ctx + s.n - 1 : s.ctx + tok, g = h / p.G;
  const int first = g * p.D + (mine ? d : 0);
  const KeyList t = key_list<32>(p.span, s.off, window_start(s.ctx, p.span.window), last);
  const long long query = s.q0 + tok, at_q = (query * p.hq + h) * p.D;
  const RowSees sees = row_sees(p.span, t, s.off, s.ctx, s.n, tok, query, p.q_pos, p.mask, p.words);
  const int io = dtype == PKV_F32 ? PKV_F32 : PKV_BF16;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  repair_elements(p.q + at_q * (io == PKV_F32 ? 4 : 2), io, mine ? d : 0, q);
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
        // (without a branch: what is not a key of this lane's dims is loaded from elsewhere and dropped)
        const bool held = on[u] && row >= 0 && mine;
        const char *k_row = p.k + (held ? row : 0), *v_row = p.v + (held ? row : 0);
        float k[E];
        repair_elements(k_row, dtype, first, k);
        repair_elements(v_row, dtype, first, v[u]);
        float sk = 1.f, sv = 1.f;
        if (dtype == PKV_I8) {
          sk = *reinterpret_cast<const float*>(k_row + p.scale_off + 4 * g);
          sv = *reinterpret_cast<const float*>(v_row + p.scale_off + 4 * g);
        }
        x[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          x[u] = fmaf(q[e], k[e], x[u]);
          v[u][e] = held ? v[u][e] * sv : 0.f;
        }
        x[u] = held ? x[u] * sk : 0.f;
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
    for (int e = 0; e < E; ++e) lost &= o[e] != o[e] || !mine;
    if (__all_sync(kWarp, lost)) break;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (!mine) return;
  if (io == PKV_F32)
    *reinterpret_cast<float4*>(p.out + (at_q + d) * 4) =
        make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
  else
    *reinterpret_cast<uint2*>(p.out + (at_q + d) * 2) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
}

}  // namespace pkv
