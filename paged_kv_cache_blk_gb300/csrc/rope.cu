// Rotary positions, fused with the append of the rotated keys.
//
// What is computed.  Pair i of a head (rotary_dim / 2 pairs) turns by the
// angle pos * f_i:  (a, b) -> (a c - b s, b c + a s), c and s scaled by the
// descriptor's attn_scale; the dims after rotary_dim pass unchanged.  The
// rotated q goes to q_out, the rotated k and v go to their slots of the pool
// (quantised for int8 pools, from the fp32 rotation: the codes are the only
// rounding), in one pass: q, k_new and v_new are read once, and nothing else
// is written.
//
// The angle.  fp32 has 24 bits: pos * f_i at position 2^20 would be off by
// 0.06 rad.  The descriptor holds each frequency as a 64-bit fraction of a
// turn instead, step = f / 2 pi * 2^64, and pos * step mod 2^64 is the angle
// modulo one turn exactly (one integer multiply); its error is that of step,
// |pos| * 2^-54 turns at most.  The top 32 bits, as a signed fraction of a half turn,
// go to sincospif, whose argument reduction is then trivial.
//
// Layout of the work.  A lane owns 8 elements (4 of fp32 up to D 128) of a head
// row, so D / EPL lanes hold one head and a warp 32 * EPL / D of them.  They
// are EPL / 2 whole pairs: adjacent elements (interleaved), or two runs
// rotary_dim / 2 apart (half layout), so no pair is split between lanes.  A warp's
// task is one token and a run of its Hq + 2 Hkv head rows: the lane's columns,
// and so its cosines and sines, are the same in every row.  The rotary_dim / 2
// angles of the token are spread over the 32 lanes, once per task, and handed
// out by shuffles.
//
// What bounds it: many tokens, the bytes of q, k and v, read and written once
// (8192 entries, Hq 32, Hkv 8, D 128, bf16: 30.8 us, 0.87 of the copy rate); into
// int8 pools, instructions and the latency of absmax chains at 20 warps an SM (6000
// tokens: 35.9 us, 18.4 M instructions, 14.6 us at full issue; 49 % of the slots used); few
// tokens, latency (the chain sequence - offset - table entry - store: 2.6 us).
#include <cmath>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "quant.cuh"
#include "slots.cuh"

namespace pkv {
namespace {

constexpr int kRopeWarps = 4;
constexpr int kRopeUnroll = 4;  // rows of a sub-warp kept in flight
constexpr unsigned kAll = 0xffffffffu;

struct RopeParams {
  char* k_cache;
  char* v_cache;
  const char* q;
  const char* k_new;
  const char* v_new;
  char* q_out;
  const int32_t* rope_pos;  // null: the token's position
  SlotSrc ss;
  long long n, num_blocks;
  long long q_stride, k_stride, v_stride, qo_stride;  // bytes from one token to the next
  int* err;
  int L, layer, bs, row_bytes, scale_off, hq, hkv;
  int rd;           // rotary_dim
  int rows_task;    // head rows of a task (a multiple of the rows a warp holds)
  int chunks;       // tasks of a token
  float attn_scale;
  unsigned long long step[PKV_ROPE_MAX_PAIRS];
};

// cos and sin of pos * f, f given as a 64-bit fraction of a turn.
__device__ __forceinline__ void rope_sincos(unsigned long long step, int pos, float scale,
                                            float* s, float* c) {
  const unsigned long long ph = step * (unsigned long long)(long long)pos;
  const int top = (int)((ph + 0x80000000ull) >> 32);
  sincospif((float)top * (1.f / 2147483648.f), s, c);
  *s *= scale;
  *c *= scale;
}

// The EPL elements of a lane as 32-bit words: two runs of EPL / 2 elements, at
// byte offsets o0 and o1 of a row (one 16-byte run where ONE).
template <typename T, int EPL, bool ONE>
__device__ __forceinline__ void load_runs(const char* row, int o0, int o1,
                                          uint32_t (&w)[EPL * sizeof(T) / 4]) {
  constexpr int W = EPL * sizeof(T) / 4;
  if constexpr (W == 4 && !ONE) {
    const uint2 a = *reinterpret_cast<const uint2*>(row + o0);
    const uint2 b = *reinterpret_cast<const uint2*>(row + o1);
    w[0] = a.x; w[1] = a.y; w[2] = b.x; w[3] = b.y;
  } else {
#pragma unroll
    for (int v = 0; v < W / 4; ++v) {
      const uint4 a = *reinterpret_cast<const uint4*>(row + (v ? o1 : o0));
      w[4 * v] = a.x; w[4 * v + 1] = a.y; w[4 * v + 2] = a.z; w[4 * v + 3] = a.w;
    }
  }
}

template <typename T, int EPL, bool ONE>
__device__ __forceinline__ void store_runs(char* row, int o0, int o1,
                                           const uint32_t (&w)[EPL * sizeof(T) / 4]) {
  constexpr int W = EPL * sizeof(T) / 4;
  if constexpr (W == 4 && !ONE) {
    *reinterpret_cast<uint2*>(row + o0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(row + o1) = make_uint2(w[2], w[3]);
  } else {
#pragma unroll
    for (int v = 0; v < W / 4; ++v)
      st_global(row + (v ? o1 : o0),
                make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]));
  }
}

template <typename T, int EPL>
__device__ __forceinline__ void unpack(const uint32_t (&w)[EPL * sizeof(T) / 4], float (&x)[EPL]) {
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    x[i] = sizeof(T) == 4 ? __uint_as_float(w[i * sizeof(T) / 4])
           : i & 1        ? bf16_hi(w[i / 2])
                          : bf16_lo(w[i / 2]);
}

template <typename T, int EPL>
__device__ __forceinline__ void pack(const float (&y)[EPL], uint32_t (&w)[EPL * sizeof(T) / 4]) {
#pragma unroll
  for (int i = 0; i < EPL * (int)sizeof(T) / 4; ++i) {
    if constexpr (sizeof(T) == 2)
      w[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
    else
      w[i] = __float_as_uint(y[i]);
  }
}

// Cosines and sines of the NF consecutive angles from f0 on.  Lane l computes
// the angles l * NPL .. l * NPL + NPL - 1 (`step`), the others come from their
// lanes.
template <int NF, int NPL>
__device__ __forceinline__ void hand_out(const unsigned long long (&step)[4], int pos, float scale,
                                         int f0, float (&s)[NF], float (&c)[NF]) {
  float ms[NPL], mc[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) rope_sincos(step[j], pos, scale, &ms[j], &mc[j]);
#pragma unroll
  for (int i = 0; i < NF; ++i) {
    s[i] = __shfl_sync(kAll, ms[i % NPL], f0 / NPL + i / NPL);
    c[i] = __shfl_sync(kAll, mc[i % NPL], f0 / NPL + i / NPL);
  }
}

enum : int { kRowQ = 0, kRowK = 1, kRowV = 2 };

// T: type of q, k_new, v_new and q_out; EPL: elements per lane; LPH: lanes per
// head row; INTER: pairs are adjacent elements; QUANT: int8 pool.
template <typename T, int EPL, int LPH, bool INTER, bool QUANT>
__global__ void __launch_bounds__(kRopeWarps * 32, 5)
    rope_append_kernel(const __grid_constant__ RopeParams p) {
  constexpr int W = EPL * sizeof(T) / 4;  // words of a lane
  constexpr int RPW = 32 / LPH;
  constexpr int NF = EPL / 2;  // pairs of a lane
  constexpr int ES = sizeof(T), ROW = EPL * LPH * ES;
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPH, col = lane % LPH;
  const bool turns = col * EPL < p.rd;
  const int half = p.rd / 2;
  const int f0 = turns ? col * NF : 0;
  // first elements of the lane's two runs
  const int e0 = INTER || !turns ? col * EPL : col * NF;
  const int e1 = INTER || !turns ? e0 + NF : e0 + half;
  const int npl = half <= 32 ? 1 : half <= 64 ? 2 : 4;
  unsigned long long step[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) step[j] = j < npl && lane * npl + j < half ? p.step[lane * npl + j] : 0;
  const int rows = p.hq + 2 * p.hkv;
  griddep_wait();
  griddep_launch_dependents();
  const long long tasks = p.n * p.chunks;
  const long long warps = (long long)gridDim.x * kRopeWarps;
  for (long long w = blockIdx.x * (long long)kRopeWarps + (threadIdx.x >> 5); w < tasks;
       w += warps) {
    const long long t = p.chunks == 1 ? w : w / p.chunks;
    const int chunk = (int)(w - t * p.chunks);
    const int r0 = chunk * p.rows_task;
    const int r1 = min(rows, r0 + p.rows_task);
    // the first rows are on their way while the chain sequence - offset - table
    // entry runs
    const int seq = ld_volatile(p.ss.tok_seq + t);
    const int pos = ld_volatile((p.rope_pos ? p.rope_pos : p.ss.tok_pos) + t);
    const int k0 = p.hq, v0 = p.hq + p.hkv;
    const char* src = r0 < k0   ? p.q + t * p.q_stride
                      : r0 < v0 ? p.k_new + t * p.k_stride - (long long)k0 * ROW
                                : p.v_new + t * p.v_stride - (long long)v0 * ROW;
    uint32_t raw[kRopeUnroll][W];
    auto fetch = [&](const char* from, int r, int end) {
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u)
        if (r + u * RPW < end)
          load_runs<T, EPL, INTER>(from + (long long)(r + u * RPW) * ROW, e0 * ES, e1 * ES, raw[u]);
    };
    if (seq >= 0) fetch(src, r0 + sub, min(r1, r0 < k0 ? k0 : r0 < v0 ? v0 : rows));
    const int64_t slot = token_slot(p.ss, t, p.num_blocks, p.bs, p.err, chunk == 0 && lane == 0);
    if (chunk == 0 && lane == 0 && p.ss.slots_out) p.ss.slots_out[t] = slot;
    if (slot < 0) continue;  // padding or out of range: nothing of this token is written
    float c[NF], s[NF];
    if (npl == 1)
      hand_out<NF, 1>(step, pos, p.attn_scale, f0, s, c);
    else if (npl == 2)
      hand_out<NF, 2>(step, pos, p.attn_scale, f0, s, c);
    else
      hand_out<NF, 4>(step, pos, p.attn_scale, f0, s, c);
    const long long dst_row =
        row_offset(slot >> (31 - __clz(p.bs)), p.layer, (int)(slot & (p.bs - 1)), p.L, p.bs,
                   p.row_bytes);

    // heads [a, b) of one kind: loads of kRopeUnroll steps (the task's first are
    // there), then stores
    bool there = true;
    auto run = [&](auto kind_tag, const char* from, int a, int b) {
      constexpr int KIND = decltype(kind_tag)::value;
#pragma unroll 1
      for (int rb = a + sub; rb - sub < b; rb += RPW * kRopeUnroll) {
        if (!there) fetch(from, rb, b);
        there = false;
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
          const int r = rb + u * RPW;
          if (r - sub >= b) break;  // (the whole warp)
          if constexpr (KIND == kRowV && !QUANT) {
            if (r < b)
              store_runs<T, EPL, INTER>(p.v_cache + dst_row + (long long)r * ROW, e0 * ES, e1 * ES,
                                        raw[u]);
            continue;
          }
          float y[EPL];
          unpack<T, EPL>(raw[u], y);
          if (KIND != kRowV && turns) {
#pragma unroll
            for (int i = 0; i < NF; ++i) {
              const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + NF;
              const float x0 = y[ia], x1 = y[ib];
              y[ia] = x0 * c[i] - x1 * s[i];
              y[ib] = x1 * c[i] + x0 * s[i];
            }
          }
          if constexpr (KIND == kRowQ || !QUANT) {
            char* dst = KIND == kRowQ ? p.q_out + t * p.qo_stride : p.k_cache + dst_row;
            uint32_t w[W];
            pack<T, EPL>(y, w);
            if (r < b)
              store_runs<T, EPL, INTER>(dst + (long long)r * ROW, e0 * ES, e1 * ES, w);
          } else {
            // absmax of the head over its LPH lanes, then scale and codes as
            // pkv_write_slots
            char* dst = (KIND == kRowK ? p.k_cache : p.v_cache) + dst_row;
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
#pragma unroll
            for (int o = LPH / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
            if (r < b) {
              const float scale = div_ieee(__uint_as_float(m), 127.f);
              uint32_t code[EPL / 4];
              quantise_bytes<EPL / 4>(y, m, scale, code);
              char* at = dst + r * (EPL * LPH);
              *reinterpret_cast<uint32_t*>(at + e0) = code[0];
              *reinterpret_cast<uint32_t*>(at + e1) = code[EPL / 4 - 1];
              if (col == 0) *reinterpret_cast<float*>(dst + p.scale_off + 4 * r) = scale;
            }
          }
        }
      }
    };
    if (r0 < k0)
      run(std::integral_constant<int, kRowQ>(), p.q + t * p.q_stride, r0, min(r1, k0));
    if (r1 > k0 && r0 < v0)
      run(std::integral_constant<int, kRowK>(), p.k_new + t * p.k_stride, max(r0, k0) - k0,
          min(r1, v0) - k0);
    if (r1 > v0)
      run(std::integral_constant<int, kRowV>(), p.v_new + t * p.v_stride, max(r0, v0) - v0, r1 - v0);
  }
}

template <typename T, int EPL, int LPH, bool QUANT>
cudaError_t launch_rope_layout(RopeParams& p, bool inter, int sms, cudaStream_t s) {
  constexpr int RPW = 32 / LPH;
  const int rows = p.hq + 2 * p.hkv;
  // Tasks of one token: as many as give every SM about 16 warps, at least one
  // warp step of rows each.
  const long long want = 16ll * sms;
  long long chunks = (want + p.n - 1) / p.n;
  const int most = (rows + RPW - 1) / RPW;
  if (chunks > most) chunks = most;
  p.rows_task = (int)((rows + chunks - 1) / chunks);
  p.rows_task = (p.rows_task + RPW - 1) / RPW * RPW;
  p.chunks = (rows + p.rows_task - 1) / p.rows_task;
  const long long ctas = (p.n * p.chunks + kRopeWarps - 1) / kRopeWarps;
  const dim3 grid((unsigned)(ctas < (1 << 30) ? ctas : (1 << 30)));
  if (inter)
    return launch_kernel(rope_append_kernel<T, EPL, LPH, true, QUANT>, grid, dim3(kRopeWarps * 32),
                         0, s, true, p);
  return launch_kernel(rope_append_kernel<T, EPL, LPH, false, QUANT>, grid, dim3(kRopeWarps * 32),
                       0, s, true, p);
}

cudaError_t launch_rope(RopeParams& p, const PoolView& v, bool inter, int sms, cudaStream_t s) {
  if (v.quant) {
    switch (v.head_dim) {
      case 32: return launch_rope_layout<__nv_bfloat16, 8, 4, true>(p, inter, sms, s);
      case 64: return launch_rope_layout<__nv_bfloat16, 8, 8, true>(p, inter, sms, s);
      case 128: return launch_rope_layout<__nv_bfloat16, 8, 16, true>(p, inter, sms, s);
      case 256: return launch_rope_layout<__nv_bfloat16, 8, 32, true>(p, inter, sms, s);
    }
  } else if (v.io_size == 2) {
    switch (v.head_dim) {
      case 32: return launch_rope_layout<__nv_bfloat16, 8, 4, false>(p, inter, sms, s);
      case 64: return launch_rope_layout<__nv_bfloat16, 8, 8, false>(p, inter, sms, s);
      case 128: return launch_rope_layout<__nv_bfloat16, 8, 16, false>(p, inter, sms, s);
      case 256: return launch_rope_layout<__nv_bfloat16, 8, 32, false>(p, inter, sms, s);
    }
  } else {
    switch (v.head_dim) {
      case 32: return launch_rope_layout<float, 4, 8, false>(p, inter, sms, s);
      case 64: return launch_rope_layout<float, 4, 16, false>(p, inter, sms, s);
      case 128: return launch_rope_layout<float, 4, 32, false>(p, inter, sms, s);
      case 256: return launch_rope_layout<float, 8, 32, false>(p, inter, sms, s);
    }
  }
  return cudaErrorInvalidValue;
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

// Frequency (radians per token) as a 64-bit fraction of a turn.
uint64_t turn_step(double f) {
  double t = f / kTwoPi;
  t -= std::floor(t);
  const double x = std::nearbyint(t * 18446744073709551616.0);  // 2^64
  return x >= 18446744073709551616.0 ? 0ull : (uint64_t)x;
}

}  // namespace
}  // namespace pkv

extern "C" {

pkv_status pkv_rope_init_freqs(pkv_rope* rope, int32_t rotary_dim, int32_t interleaved,
                               const double* inv_freq, double attn_scale) {
  if (!rope || !inv_freq || rotary_dim <= 0 || rotary_dim % 2 != 0) return PKV_ERR_INVALID_ARG;
  if (rotary_dim > 2 * PKV_ROPE_MAX_PAIRS) return PKV_ERR_UNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return PKV_ERR_INVALID_ARG;
  if (!std::isfinite(attn_scale) || !(std::fabs(attn_scale) <= 3.0e38)) return PKV_ERR_INVALID_ARG;
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (!std::isfinite(inv_freq[i])) return PKV_ERR_INVALID_ARG;
  std::memset(rope, 0, sizeof(*rope));
  rope->rotary_dim = rotary_dim;
  rope->interleaved = interleaved;
  rope->attn_scale = (float)attn_scale;
  for (int i = 0; i < rotary_dim / 2; ++i) rope->step[i] = pkv::turn_step(inv_freq[i]);
  return PKV_OK;
}

pkv_status pkv_rope_init(pkv_rope* rope, int32_t rotary_dim, int32_t interleaved, double base,
                         int32_t scaling, double factor, double original_len, double turns_fast,
                         double turns_slow) {
  if (!rope || rotary_dim <= 0 || rotary_dim % 2 != 0) return PKV_ERR_INVALID_ARG;
  if (rotary_dim > 2 * PKV_ROPE_MAX_PAIRS) return PKV_ERR_UNSUPPORTED;
  if (!std::isfinite(base) || !(base > 0.0)) return PKV_ERR_INVALID_ARG;
  if (scaling < PKV_ROPE_PLAIN || scaling > PKV_ROPE_BY_PARTS) return PKV_ERR_INVALID_ARG;
  if (scaling != PKV_ROPE_PLAIN && (!std::isfinite(factor) || !(factor >= 1.0)))
    return PKV_ERR_INVALID_ARG;
  if (scaling == PKV_ROPE_BASE) {
    if (rotary_dim <= 2) return PKV_ERR_INVALID_ARG;
    base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
  }
  double attn = 1.0;
  if (scaling == PKV_ROPE_BY_PARTS) {
    if (!std::isfinite(original_len) || !(original_len > 0.0) || !std::isfinite(turns_fast) ||
        !std::isfinite(turns_slow) || !(turns_fast > turns_slow))
      return PKV_ERR_INVALID_ARG;
    attn = 0.1 * std::log(factor) + 1.0;
  }
  double f[PKV_ROPE_MAX_PAIRS];
  for (int i = 0; i < rotary_dim / 2; ++i) {
    f[i] = std::pow(base, -2.0 * i / rotary_dim);
    if (scaling == PKV_ROPE_LINEAR) f[i] /= factor;
    if (scaling == PKV_ROPE_BY_PARTS) {
      const double turns = original_len * f[i] / pkv::kTwoPi;
      double keep = (turns - turns_slow) / (turns_fast - turns_slow);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f[i] = keep * f[i] + (1.0 - keep) * f[i] / factor;
    }
  }
  return pkv_rope_init_freqs(rope, rotary_dim, interleaved, f, attn);
}

pkv_status pkv_rope_append(const pkv_pool* pool, int32_t layer, const pkv_rope* rope,
                           const int32_t* block_tables, int32_t max_blocks_per_seq,
                           const int32_t* offsets, int32_t batch, const int32_t* token_seq,
                           const int32_t* token_pos, const int32_t* rope_pos, int64_t num_tokens,
                           const void* q, int64_t q_stride, int32_t num_q_heads,
                           const void* k_new, int64_t k_stride, const void* v_new,
                           int64_t v_stride, void* q_out, int64_t q_out_stride,
                           int64_t* slot_mapping, cudaStream_t stream) {
  pkv::PoolView v;
  int st = pkv::pool_view(pool, true, &v);
  if (st != PKV_OK) return (pkv_status)st;
  if (!rope || layer < 0 || layer >= v.num_layers || num_tokens < 0 || batch < 0 ||
      num_q_heads < 0)
    return PKV_ERR_INVALID_ARG;
  if (rope->rotary_dim <= 0 || rope->rotary_dim % 2 != 0 || rope->rotary_dim > v.head_dim ||
      (rope->interleaved != 0 && rope->interleaved != 1) || !std::isfinite(rope->attn_scale))
    return PKV_ERR_INVALID_ARG;
  if (v.head_dim != 32 && v.head_dim != 64 && v.head_dim != 128 && v.head_dim != 256)
    return PKV_ERR_UNSUPPORTED;
  // a lane's elements turn together
  const int piece = v.io_size == 4 && v.head_dim <= 128 ? 4 : 8;
  if (rope->rotary_dim % piece != 0) return PKV_ERR_UNSUPPORTED;
  if (num_q_heads > (1 << 20)) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!token_seq || !token_pos || !k_new || !v_new) return PKV_ERR_INVALID_ARG;
  if (num_q_heads > 0 && (!q || !q_out)) return PKV_ERR_INVALID_ARG;
  if (batch > 0 && (!block_tables || max_blocks_per_seq <= 0)) return PKV_ERR_INVALID_ARG;
  if (!pkv::aligned(token_seq, 4) || !pkv::aligned(token_pos, 4) || !pkv::aligned(rope_pos, 4) ||
      !pkv::aligned(block_tables, 4) || !pkv::aligned(offsets, 4) ||
      !pkv::aligned(slot_mapping, 8) || !pkv::aligned(q, 16) || !pkv::aligned(q_out, 16) ||
      !pkv::aligned(k_new, 16) || !pkv::aligned(v_new, 16))
    return PKV_ERR_INVALID_ARG;
  const int64_t kv_row = (int64_t)v.num_kv_heads * v.head_dim;
  const int64_t q_row = (int64_t)num_q_heads * v.head_dim;
  const int64_t unit = 16 / v.io_size;
  const int64_t most = INT64_MAX / 16 / num_tokens;  // keeps every byte offset in 64 bits
  for (int64_t x : {q_stride, k_stride, v_stride, q_out_stride})
    if (x % unit != 0 || x > most) return PKV_ERR_INVALID_ARG;
  if (k_stride < kv_row || v_stride < kv_row) return PKV_ERR_INVALID_ARG;
  if (num_q_heads > 0 && (q_stride < q_row || q_out_stride < q_row)) return PKV_ERR_INVALID_ARG;
  int optin, grid, validate, sms;
  int* err;
  if ((st = pkv::device_facts(&optin, &err, &grid, &validate)) != PKV_OK) return (pkv_status)st;
  if ((st = pkv::device_sm_count(&sms)) != PKV_OK) return (pkv_status)st;
  if (validate) {
    if ((st = pkv::clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
    if ((st = pkv::launch_status(pkv::launch_validate_tokens(
             v, block_tables, max_blocks_per_seq, offsets, batch, token_seq, token_pos,
             num_tokens, err, stream))) != PKV_OK)
      return (pkv_status)st;
    if ((st = pkv::read_and_clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
  }
  pkv::RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.k_cache = v.k_mut;
  p.v_cache = v.v_mut;
  p.q = static_cast<const char*>(q);
  p.k_new = static_cast<const char*>(k_new);
  p.v_new = static_cast<const char*>(v_new);
  p.q_out = static_cast<char*>(q_out);
  p.rope_pos = rope_pos;
  p.ss = pkv::SlotSrc{nullptr, block_tables, offsets, token_seq, token_pos, slot_mapping,
                      max_blocks_per_seq, batch};
  p.n = num_tokens;
  p.num_blocks = v.num_blocks;
  p.q_stride = q_stride * v.io_size;
  p.k_stride = k_stride * v.io_size;
  p.v_stride = v_stride * v.io_size;
  p.qo_stride = q_out_stride * v.io_size;
  p.err = err;
  p.L = v.num_layers;
  p.layer = layer;
  p.bs = v.block_size;
  p.row_bytes = v.row_bytes;
  p.scale_off = v.scale_off;
  p.hq = num_q_heads;
  p.hkv = v.num_kv_heads;
  p.rd = rope->rotary_dim;
  p.attn_scale = rope->attn_scale;
  for (int i = 0; i < rope->rotary_dim / 2; ++i) p.step[i] = rope->step[i];
  if ((st = pkv::launch_status(pkv::launch_rope(p, v, rope->interleaved != 0, sms, stream))) !=
      PKV_OK)
    return (pkv_status)st;
  return validate ? (pkv_status)pkv::read_and_clear_error_word(err, stream) : PKV_OK;
}

}  // extern "C"
