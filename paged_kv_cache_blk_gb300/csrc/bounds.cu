// Key bounds of the blocks that hold new tokens (pkv_update_block_bounds; see
// bounds.cuh for what they are).
//
// The rows of a block are read in place: D / EPL lanes own one (block, kv
// head), EPL elements (16 bytes) each, and step down the rows, consecutive
// heads in consecutive lanes, so a warp reads whole 512-byte runs of token
// rows.  The running extremes stay in the type of the pool (packed bf16
// maxima; fp32 products code * scale for int8 pools).  Every row from 0 to
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
      const int c = (int)((w[i / 4] >> (8 * (i % 4))) & 0xFFu) - 128;
      const float x = mul_ieee((float)c, scale);
      hi[i] = max_nan(hi[i], x);
      lo[i] = min_nan(lo[i], x);
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
  constexpr int GROUPS = kBoundThreads / LPH;  // (block, head) pairs of a CTA
  constexpr int UNROLL = 8;
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
  const int items = nj * p.hkv;  // (mb * hkv is checked)
  const int col = threadIdx.x % LPH;
  const int step = p.ctas_seq * GROUPS;
  const int32_t* table = p.bt + (long long)b * p.mb + j0;
  int it = x * GROUPS + (int)threadIdx.x / LPH;
  int blk = it < items ? table[it / p.hkv] : -1;
  // groups of a warp run the same number of steps, so the shuffles stay whole
  for (int i0 = x * GROUPS; i0 < items; i0 += step) {
    const bool live = it < items;
    const int j = j0 + (live ? it / p.hkv : 0);
    const int g = live ? it % p.hkv : 0;
    const int mine = blk;
    it = it < items - step ? it + step : items;
    blk = it < items ? table[it / p.hkv] : -1;  // the next step's, ahead of its rows
    const bool ok = live && mine >= 0 && mine < p.num_blocks;
    if (live && !ok && col == 0) set_error(p.err, kErrIndex);
    const int rows = ok ? min(p.bs, end - j * p.bs) : 0;
    const char* src = p.k + row_offset(ok ? mine : 0, p.layer, 0, p.L, p.bs, p.row_bytes);
    const char* elems = src + (long long)(g * LPH + col) * 16;
    const char* unit = src + p.scale_off + 4 * g;
    Extremes<MODE, EPL> ex;
    ex.init();
    int r = 0;
    for (; r + UNROLL <= rows; r += UNROLL) {
      uint4 v[UNROLL];
      float s[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        v[u] = ld_stream(elems + (long long)(r + u) * p.row_bytes);
        s[u] = MODE == PKV_I8
                   ? *reinterpret_cast<const float*>(unit + (long long)(r + u) * p.row_bytes)
                   : 0.f;
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) ex.add(v[u], s[u]);
    }
    for (; r < rows; ++r)
      ex.add(ld_stream(elems + (long long)r * p.row_bytes),
             MODE == PKV_I8 ? *reinterpret_cast<const float*>(unit + (long long)r * p.row_bytes)
                            : 0.f);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      m = max(m, max(__float_as_uint(ex.top(i)) & 0x7FFFFFFFu,
                     __float_as_uint(ex.bottom(i)) & 0x7FFFFFFFu));
#pragma unroll
    for (int o = LPH / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
    if (!ok) continue;
    const int e = bound_exponent(m);
    const float inv = pow2f(-e);
    uint32_t hw[EPL / 4] = {}, lw[EPL / 4] = {};
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      hw[i / 4] |= (uint32_t)(code_up(ex.top(i), inv) + 128) << (8 * (i % 4));
      lw[i / 4] |= (uint32_t)(code_down(ex.bottom(i), inv) + 128) << (8 * (i % 4));
    }
    const long long head = ((long long)mine * p.L + p.layer) * p.hkv + g;
    char* dst = p.codes + head * (2 * D) + col * EPL;
    store_bytes(dst, hw);
    store_bytes(dst + D, lw);
    if (col == 0) p.scales[head] = pow2f(e);
  }
}

template <int MODE>
cudaError_t launch_bounds_mode(BoundParams& p, int d, int batch, int sms, cudaStream_t s) {
  // Enough CTAs to fill the SMs over the batch (48 warps each), none that the
  // longest possible table would leave idle.
  const int lph = d / (MODE == PKV_BF16 ? 8 : MODE == PKV_F32 ? 4 : 16);
  const long long groups = kBoundThreads / lph;
  long long ctas = ((long long)p.mb * p.hkv + groups - 1) / groups;
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
  // table positions and (block, head) pairs are 32-bit in the kernel
  if ((int64_t)max_blocks_per_seq * v.block_size > INT32_MAX || batch > (1 << 24) ||
      (int64_t)max_blocks_per_seq * v.num_kv_heads > INT32_MAX / 2)
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
