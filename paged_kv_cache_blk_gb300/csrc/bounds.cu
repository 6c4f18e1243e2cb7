// Key bounds of the blocks that hold new tokens (pkv_update_block_bounds; see
// bounds.cuh for what they are).
//
// The rows of a block are read in place.  A warp owns one (block, kv head):
// D / EPL lanes hold a row, EPL elements (16 bytes) each, and the 32 EPL / D
// groups of them take every so-manieth row, so that a single block, as after a
// decode step, is not one long chain of loads.  The running extremes stay in
// the type of the pool (packed bf16 maxima; fp32 products code * scale for int8
// pools), and are merged over the groups by shuffles.  Every row from 0 to
// the last one the sequence holds counts, the rows before a first-block
// offset too: they belong to a prefix shared with other sequences, and all
// holders of a full block then store the same bytes.
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

// Extremes of EPL elements, stepping down rows.
template <int MODE, int EPL>
struct Extremes;

template <int EPL>
struct Extremes<PKV_BF16, EPL> {  // EPL = 8, packed pairs
  uint32_t hi[4], lo[4];
  __device__ void init() {
#pragma unroll
    for (int i = 0; i < 4; ++i) { hi[i] = 0xFF80FF80u; lo[i] = 0x7F807F80u; }
  }
  __device__ void add(const uint4& r, float) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(hi[i]) : "r"(w[i]));
      asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(lo[i]) : "r"(w[i]));
    }
  }
  __device__ void merge(int o) {  // with the lane `o` away
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = __shfl_xor_sync(kAll, hi[i], o), b = __shfl_xor_sync(kAll, lo[i], o);
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(hi[i]) : "r"(a));
      asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(lo[i]) : "r"(b));
    }
  }
  __device__ float top(int i) const { return i & 1 ? bf16_hi(hi[i / 2]) : bf16_lo(hi[i / 2]); }
  __device__ float bottom(int i) const { return i & 1 ? bf16_hi(lo[i / 2]) : bf16_lo(lo[i / 2]); }
};

template <int EPL>
struct Extremes<PKV_F32, EPL> {  // EPL = 4
  float hi[4], lo[4];
  __device__ void init() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = __uint_as_float(0xFF800000u);
      lo[i] = __uint_as_float(0x7F800000u);
    }
  }
  __device__ void add(const uint4& r, float) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = max_nan(hi[i], __uint_as_float(w[i]));
      lo[i] = min_nan(lo[i], __uint_as_float(w[i]));
    }
  }
  __device__ void merge(int o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = max_nan(hi[i], __shfl_xor_sync(kAll, hi[i], o));
      lo[i] = min_nan(lo[i], __shfl_xor_sync(kAll, lo[i], o));
    }
  }
  __device__ float top(int i) const { return hi[i]; }
  __device__ float bottom(int i) const { return lo[i]; }
};

template <int EPL>
struct Extremes<PKV_I8, EPL> {  // EPL = 16 codes
  float hi[16], lo[16];
  __device__ void init() {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      hi[i] = __uint_as_float(0xFF800000u);
      lo[i] = __uint_as_float(0x7F800000u);
    }
  }
  __device__ void add(const uint4& r, float scale) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      // the byte as the low mantissa bits of 2^23, less 2^23 + 128
      const float c = __uint_as_float(__byte_perm(w[i / 4], 0x4B000000u, 0x7540 | (i % 4))) -
                      8388736.f;
      const float x = mul_ieee(c, scale);
      hi[i] = max_nan(hi[i], x);
      lo[i] = min_nan(lo[i], x);
    }
  }
  __device__ void merge(int o) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      hi[i] = max_nan(hi[i], __shfl_xor_sync(kAll, hi[i], o));
      lo[i] = min_nan(lo[i], __shfl_xor_sync(kAll, lo[i], o));
    }
  }
  __device__ float top(int i) const { return hi[i]; }
  __device__ float bottom(int i) const { return lo[i]; }
};

template <int N>
__device__ __forceinline__ void store_bytes(char* dst, const uint32_t (&w)[N]) {
  if constexpr (N == 4)
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (N == 2)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = w[0];
}

template <int MODE, int D>
__global__ void __launch_bounds__(kBoundThreads) update_bounds_kernel(const BoundParams p) {
  constexpr int EPL = MODE == PKV_BF16 ? 8 : MODE == PKV_F32 ? 4 : 16;
  constexpr int LPH = D / EPL;
  constexpr int RPW = 32 / LPH;                // rows a warp reads at once
  constexpr int WARPS = kBoundThreads / 32;    // (block, head) pairs of a CTA
  constexpr int UNROLL = MODE == PKV_I8 ? 4 : 8;
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
    Extremes<MODE, EPL> ex;
    ex.init();
    for (int r = sub; r < rows; r += RPW * UNROLL) {
      uint4 v[UNROLL];
      float s[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        // past the end, the last row again; a block is less than 4 GB
        const uint32_t at = (uint32_t)min(r + u * RPW, rows - 1) * (uint32_t)p.row_bytes;
        v[u] = ld_stream(elems + at);
        s[u] = MODE == PKV_I8 ? *reinterpret_cast<const float*>(unit + at) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) ex.add(v[u], s[u]);
    }
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1) ex.merge(o);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      m = max(m, max(__float_as_uint(ex.top(i)) & 0x7FFFFFFFu,
                     __float_as_uint(ex.bottom(i)) & 0x7FFFFFFFu));
#pragma unroll
    for (int o = LPH / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
    const int e = bound_exponent(m);
    const float inv = pow2f(-e);
    const long long at = ((long long)mine * p.L + p.layer) * p.hkv + head;
    char* dst = p.codes + at * (2 * D) + col * EPL;
    // every group of lanes holds the result: one writes hi, another lo
    if (sub == 0) {
      uint32_t w[EPL / 4] = {};
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        w[i / 4] |= (uint32_t)(code_up(ex.top(i), inv) + 128) << (8 * (i % 4));
      store_bytes(dst, w);
      if (col == 0) p.scales[at] = pow2f(e);
    }
    if (sub == (RPW > 1 ? 1 : 0)) {
      uint32_t w[EPL / 4] = {};
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        w[i / 4] |= (uint32_t)(code_down(ex.bottom(i), inv) + 128) << (8 * (i % 4));
      store_bytes(dst + D, w);
    }
  }
}

template <int MODE>
cudaError_t launch_bounds_mode(BoundParams& p, int d, int batch, int sms, cudaStream_t s) {
  // Enough CTAs to fill the SMs over the batch (48 warps each), none that the
  // longest possible table would leave idle.
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

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

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
