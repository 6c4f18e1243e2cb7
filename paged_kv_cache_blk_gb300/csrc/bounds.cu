// Key bounds of the blocks that hold new tokens (pkv_update_block_bounds; see
// bounds.cuh for what they are).
//
// The rows of a block are read in place.  A warp owns one (block, kv head):
// D / EPL lanes hold a row, EPL elements (16 bytes) each, and the 32 EPL / D
// groups of them take the rows in turn, so that a single block, as after a
// decode step, is not one long chain of loads.  The running extremes stay in
// the type of the pool (packed bf16 maxima; fp32 products code * scale for int8
// pools), and are merged over the groups so that each lane ends up with, and
// codes, its own part of them.  Every row from 0 to the last one the sequence
// holds counts, the rows before a first-block offset too: they belong to a
// prefix shared with other sequences, and all holders of a full block then
// store the same bytes.
//
// What bounds it: the keys' bytes for bf16 and fp32 pools (73K prompt tokens, Hkv
// 8, D 128: 29.2 us, 5.7 TB/s; fp32 43.5 us, 6.1 TB/s).  int8 (38.9 us, 1.9 TB/s): 25 M
// instructions, 20 us at full issue, most of them (permutes, maxima, minima) on the
// ALU pipe, 66 % of its cycles busy, at 14 warps an SM (104 registers allow 16).  Four
// heads a warp, without the merge, took 29.4 us in bf16 but 28.6 us instead of 6.1
// for the last blocks of 20 sequences in int8.
#include "bounds.cuh"
#include "common.cuh"
#include "slots.cuh"

namespace pkv {
namespace {

constexpr int kBoundThreads = 128;
constexpr unsigned kAll = 0xffffffffu;

struct BoundParams {
  const char* k;
  char* codes;
  float* scales;
  const int32_t* bt;
  const int32_t* lens;
  const int32_t* offs;
  const int32_t* first;  // null: every block
  long long num_blocks;
  int* err;
  int mb, bs, L, layer, hkv, row_bytes, scale_off;
  int ctas_seq;  // CTAs of one sequence
};

// Running extremes of a lane's EPL elements: W words of PER elements each.
template <int MODE>
struct Extremes {
  static constexpr int W = MODE == PKV_I8 ? 16 : 4, PER = MODE == PKV_BF16 ? 2 : 1;
  uint32_t hi[W], lo[W];

  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (MODE == PKV_BF16) {
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
      return a;
    }
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) {
    if constexpr (MODE == PKV_BF16) {
      asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
      return a;
    }
    return __float_as_uint(min_nan(__uint_as_float(a), __uint_as_float(b)));
  }

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      hi[i] = MODE == PKV_BF16 ? 0xFF80FF80u : 0xFF800000u;
      lo[i] = MODE == PKV_BF16 ? 0x7F807F80u : 0x7F800000u;
    }
  }

  __device__ __forceinline__ void add(const uint4& r, float scale) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < W; ++i) {
      uint32_t x = w[i % 4];
      if constexpr (MODE == PKV_I8) {
        // the byte as the low mantissa bits of 2^23, less 2^23 + 128
        const float c = __uint_as_float(__byte_perm(w[i / 4], 0x4B000000u, 0x7540 | (i % 4))) -
                        8388736.f;
        x = __float_as_uint(mul_ieee(c, scale));
      }
      hi[i] = larger(hi[i], x);
      lo[i] = smaller(lo[i], x);
    }
  }

  // Merge with the lanes o, 2 o, .. 16 away: at each step a lane keeps half of
  // its words and gets its partner's part of them, so that in the end each
  // holds its own N words of the result, hi[0..N) and lo[0..N).  Returns the
  // first element among the lane's EPL.
  template <int O, int N = W>
  __device__ __forceinline__ int scatter(int lane) {
    if constexpr (O < 32) {
      constexpr int H = N / 2;
      const bool upper = lane & O;
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const uint32_t gh = __shfl_xor_sync(kAll, upper ? hi[k] : hi[k + H], O);
        const uint32_t gl = __shfl_xor_sync(kAll, upper ? lo[k] : lo[k + H], O);
        hi[k] = larger(upper ? hi[k + H] : hi[k], gh);
        lo[k] = smaller(upper ? lo[k + H] : lo[k], gl);
      }
      return (upper ? H * PER : 0) + scatter<2 * O, H>(lane);
    }
    return 0;
  }

  __device__ __forceinline__ float top(int i) const { return value(hi, i); }
  __device__ __forceinline__ float bottom(int i) const { return value(lo, i); }

 private:
  __device__ __forceinline__ float value(const uint32_t (&w)[W], int i) const {
    if constexpr (MODE == PKV_BF16) return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    return __uint_as_float(w[i]);
  }
};

template <int MODE, int D>
__global__ void __launch_bounds__(kBoundThreads) update_bounds_kernel(const BoundParams p) {
  constexpr int EPL = MODE == PKV_BF16 ? 8 : MODE == PKV_F32 ? 4 : 16;
  constexpr int LPH = D / EPL;
  constexpr int RPW = 32 / LPH;                // rows a warp reads at once
  constexpr int WARPS = kBoundThreads / 32;    // (block, head) pairs of a CTA
  constexpr int UNROLL = RPW < 2 ? 8 : 16 / RPW;  // steps of a block of 16 rows
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / p.ctas_seq, x = blockIdx.x % p.ctas_seq;
  const int len = p.lens[b], off = p.offs ? p.offs[b] : 0;
  if (len < 0 || off < 0 || off >= p.bs || (long long)off + len > (long long)p.mb * p.bs) {
    if (x == 0 && threadIdx.x == 0) set_error(p.err, kErrCapacity);
    return;
  }
  const int first = p.first ? max(p.first[b], 0) : 0;
  if (first >= len) return;
  const int end = off + len;  // table positions held: below 2^31 (mb * bs is checked)
  const int j0 = (off + first) / p.bs;
  const int nj = (end - 1) / p.bs + 1 - j0;
  const int lane = threadIdx.x & 31;
  const int col = lane % LPH, sub = lane / LPH;
  const int step = p.ctas_seq * WARPS;
  const int step_j = step / p.hkv, step_g = step - step_j * p.hkv;
  const int32_t* table = p.bt + (long long)b * p.mb + j0;
  const int first_it = x * WARPS + (int)threadIdx.x / 32;
  int j = first_it / p.hkv, g = first_it - j * p.hkv;  // blocks from j0 on
  int blk = j < nj ? table[j] : -1;
  while (j < nj) {
    const int mine = blk, head = g, rows = min(p.bs, end - (j0 + j) * p.bs);
    j += step_j;
    g += step_g;
    if (g >= p.hkv) { g -= p.hkv; ++j; }
    blk = j < nj ? table[j] : -1;  // the next one's, ahead of its rows
    if (mine < 0 || mine >= p.num_blocks) {
      if (lane == 0) set_error(p.err, kErrIndex);
      continue;
    }
    const char* src = p.k + row_offset(mine, p.layer, 0, p.L, p.bs, p.row_bytes);
    const char* elems = src + (long long)(head * LPH + col) * 16;
    const char* unit = src + p.scale_off + 4 * head;
    Extremes<MODE> ex;
    ex.init();
    for (int r = sub; r < rows; r += RPW * UNROLL) {
      uint4 v[UNROLL];
      float s[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        if (r + u * RPW >= rows) break;
        const uint32_t at = (uint32_t)(r + u * RPW) * (uint32_t)p.row_bytes;  // (checked)
        v[u] = ld_stream(elems + at);
        s[u] = MODE == PKV_I8 ? *reinterpret_cast<const float*>(unit + at) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        if (r + u * RPW >= rows) break;
        ex.add(v[u], s[u]);
      }
    }
    constexpr int N = EPL / RPW;  // elements whose result this lane ends up with
    const int d = col * EPL + ex.template scatter<LPH>(lane);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      m = max(m, max(__float_as_uint(ex.top(i)) & 0x7FFFFFFFu,
                     __float_as_uint(ex.bottom(i)) & 0x7FFFFFFFu));
    m = __reduce_max_sync(kAll, m);
    const int e = bound_exponent(m);
    const float inv = pow2f(-e);
    const long long at = ((long long)mine * p.L + p.layer) * p.hkv + head;
    uint32_t hw = 0, lw = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      hw |= (uint32_t)(code_up(ex.top(i), inv) + 128) << (8 * i);
      lw |= (uint32_t)(code_down(ex.bottom(i), inv) + 128) << (8 * i);
    }
    char* dst = p.codes + at * (2 * D) + d;
    if constexpr (N == 4) {
      *reinterpret_cast<uint32_t*>(dst) = hw;
      *reinterpret_cast<uint32_t*>(dst + D) = lw;
    } else {
      *reinterpret_cast<uint16_t*>(dst) = (uint16_t)hw;
      *reinterpret_cast<uint16_t*>(dst + D) = (uint16_t)lw;
    }
    if (lane == 0) p.scales[at] = pow2f(e);
  }
}

template <int MODE>
cudaError_t launch_bounds_mode(BoundParams& p, int d, int batch, int sms, cudaStream_t s) {
  // 12 CTAs an SM over the batch, two to three times what it holds at once (4 of 104
  // registers for int8, 5 of 96 for bf16, D 128), so that the CTAs of long sequences
  // find room behind those of short ones; none that the longest possible table
  // would leave idle.  Prompts of 512 to 4096 tokens, 32 sequences: with 5 34.5 us, with
  // 10 30.1, 12 29.2, 20 28.6 (int8 47.8, 39.9, 38.9, 37.2); their last blocks alone, bs 16
  // (int8): 3.6, 4.4, 4.7, 5.9.
  const long long warps = kBoundThreads / 32;
  long long ctas = ((long long)p.mb * p.hkv + warps - 1) / warps;
  const long long want = (12ll * sms + batch - 1) / batch;
  if (ctas > want) ctas = want;
  p.ctas_seq = (int)ctas;
  const dim3 grid((unsigned)(ctas * batch));
  if (d == 64)
    return launch_kernel(update_bounds_kernel<MODE, 64>, grid, dim3(kBoundThreads), 0, s, true, p);
  return launch_kernel(update_bounds_kernel<MODE, 128>, grid, dim3(kBoundThreads), 0, s, true, p);
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_update_block_bounds(const pkv_pool* pool, int32_t layer,
                                              const int32_t* block_tables,
                                              int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                              const int32_t* offsets, const int32_t* first_pos,
                                              int32_t batch, void* bound_codes,
                                              float* bound_scales, cudaStream_t stream) {
  pkv::PoolView v;
  int st = pkv::pool_view(pool, true, &v);
  if (st != PKV_OK) return (pkv_status)st;
  if (layer < 0 || layer >= v.num_layers || batch < 0) return PKV_ERR_INVALID_ARG;
  if (v.head_dim != 64 && v.head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (batch == 0) return PKV_OK;
  if (!block_tables || max_blocks_per_seq <= 0 || !seq_lens || !bound_codes || !bound_scales)
    return PKV_ERR_INVALID_ARG;
  if (!pkv::aligned(block_tables, 4) || !pkv::aligned(seq_lens, 4) || !pkv::aligned(offsets, 4) ||
      !pkv::aligned(first_pos, 4) || !pkv::aligned(bound_codes, 16) ||
      !pkv::aligned(bound_scales, 4))
    return PKV_ERR_INVALID_ARG;
  // table positions and offsets within a block are 32-bit in the kernel
  if ((int64_t)max_blocks_per_seq * v.block_size > INT32_MAX || batch > (1 << 24) ||
      (int64_t)v.block_size * v.row_bytes > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  int optin, grid, validate, sms;
  int* err;
  if ((st = pkv::device_facts(&optin, &err, &grid, &validate)) != PKV_OK) return (pkv_status)st;
  if ((st = pkv::device_sm_count(&sms)) != PKV_OK) return (pkv_status)st;
  if (validate) {
    if ((st = pkv::clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
    if ((st = pkv::launch_status(pkv::launch_validate_tables(
             v, block_tables, max_blocks_per_seq, seq_lens, offsets, batch, nullptr, 0, err,
             stream))) != PKV_OK)
      return (pkv_status)st;
    if ((st = pkv::read_and_clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
  }
  pkv::BoundParams p;
  p.k = v.k;
  p.codes = static_cast<char*>(bound_codes);
  p.scales = bound_scales;
  p.bt = block_tables;
  p.lens = seq_lens;
  p.offs = offsets;
  p.first = first_pos;
  p.num_blocks = v.num_blocks;
  p.err = err;
  p.mb = max_blocks_per_seq;
  p.bs = v.block_size;
  p.L = v.num_layers;
  p.layer = layer;
  p.hkv = v.num_kv_heads;
  p.row_bytes = v.row_bytes;
  p.scale_off = v.scale_off;
  const cudaError_t e =
      v.quant ? pkv::launch_bounds_mode<PKV_I8>(p, v.head_dim, batch, sms, stream)
      : v.io_size == 2 ? pkv::launch_bounds_mode<PKV_BF16>(p, v.head_dim, batch, sms, stream)
                       : pkv::launch_bounds_mode<PKV_F32>(p, v.head_dim, batch, sms, stream);
  if ((st = pkv::launch_status(e)) != PKV_OK) return (pkv_status)st;
  return validate ? (pkv_status)pkv::read_and_clear_error_word(err, stream) : PKV_OK;
}
