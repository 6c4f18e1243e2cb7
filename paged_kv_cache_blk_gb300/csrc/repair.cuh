// Results that a value which their query does not see has spoiled.
//
// The kernels multiply a tile's V rows by the weights of several queries at once, 0 where a
// query does not see a row; 0 times an infinity or a NaN is NaN.  A result that came out NaN or
// infinite although its weights' sum is finite (scores of seen keys decide that sum alone) is
// computed again by the thread that wrote it, over the seen keys only.  Off the usual path: no
// speed is sought, and the call takes few values so that the kernels keep theirs in registers.
#pragma once

#include "common.cuh"
#include "span.cuh"

namespace pkv {

__device__ __forceinline__ bool nonfinite(float x) { return (__float_as_uint(x) << 1) >= 0xff000000u; }

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

__device__ __forceinline__ float repair_element(const char* row, int dtype, int i, float scale) {
  if (dtype == PKV_F32) return reinterpret_cast<const float*>(row)[i];
  if (dtype == PKV_BF16)
    return __uint_as_float((uint32_t) reinterpret_cast<const unsigned short*>(row)[i] << 16);
  return ((float)reinterpret_cast<const unsigned char*>(row)[i] - 128.f) * scale;
}

// Dims d0 .. d0 + n - 1 of the result of token tok and query head h of sequence b, kAtOnce of
// them at a time, in registers.
template <int kAtOnce>
static __device__ __noinline__ void repair_query(const Repair& p, int b, int tok, int h, int d0,
                                                 int n) {
  const SeqSpan s = seq_span(p.span, b);
  const int last = p.mask ? s.ctx + s.n - 1 : s.ctx + tok, g = h / p.G;
  const KeyList t = key_list<32>(p.span, s.off, window_start(s.ctx, p.span.window), last);
  const long long query = s.q0 + tok, at_q = (query * p.hq + h) * p.D;
  const RowSees sees = row_sees(p.span, t, s.off, s.ctx, s.n, tok, query, p.q_pos, p.mask, p.words);
  const int io = p.dtype == PKV_F32 ? PKV_F32 : PKV_BF16, first = g * p.D;
  const char* q = p.q + at_q * (io == PKV_F32 ? 4 : 2);
  for (int end = d0 + n; d0 < end; d0 += kAtOnce) {
    float o[kAtOnce], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int d = 0; d < kAtOnce; ++d) o[d] = 0.f;
    for (int x0 = 0; x0 < t.nt * 32; x0 += 32) {
      for (uint32_t w = sees.bits_from(x0); w; w &= w - 1) {
        const int pos = t.position(x0 + __ffs(w) - 1);
        const int blk = p.bt[(long long)b * p.span.mb + (pos >> p.bs_bits)];
        const bool held = blk >= 0 && blk < p.num_blocks;  // others read as zeros
        const long long at =
            held ? ((((long long)blk * p.L + p.layer) << p.bs_bits) + (pos & ((1 << p.bs_bits) - 1))) *
                       p.row_bytes
                 : 0;
        float sk = 1.f, sv = 1.f, x = 0.f;
        if (p.dtype == PKV_I8) {
          sk = *reinterpret_cast<const float*>(p.k + at + p.scale_off + 4 * g);
          sv = *reinterpret_cast<const float*>(p.v + at + p.scale_off + 4 * g);
        }
        if (held) {
          for (int d = 0; d < p.D; ++d)
            x = fmaf(repair_element(q, io, d, 1.f), repair_element(p.k + at, p.dtype, first + d, sk), x);
        }
        x *= p.qscale;
        const float top = fmaxf(m, x), shrink = m == -INFINITY ? 0.f : exp2f(m - top);
        const float e = x == -INFINITY ? 0.f : exp2f(x - top);
        m = top;
        l = l * shrink + e;
#pragma unroll
        for (int d = 0; d < kAtOnce; ++d) {
          const bool on = held && d0 + d < end;
          const float y = on ? repair_element(p.v + at, p.dtype, first + d0 + d, sv) : 0.f;
          o[d] = fmaf(e, y, o[d] * shrink);
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int d = 0; d < kAtOnce; ++d) {
      if (d0 + d >= end) break;
      const long long i = at_q + d0 + d;
      if (io == PKV_F32)
        reinterpret_cast<float*>(p.out)[i] = o[d] * inv;
      else
        reinterpret_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16(o[d] * inv);
    }
  }
}

}  // namespace pkv
