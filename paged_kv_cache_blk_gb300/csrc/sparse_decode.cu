// Sparse paged decode attention (pkv_decode_attention_sparse): attention of
// each query over the blocks selected for it, per kv head.
//
// What is computed.  For query token t (sequence b, position P) and query
// head h of kv head g: softmax attention over the tokens i <= P of the blocks
// that the list of (t, g) names, K and V read in place through the table.
//
// What bounds it: the K and V bytes of the selected blocks, one head of each
// row (256 bytes for bf16, D 128), read once for the G heads of the group.
//
// How.  A cluster of CTAs per (t, g); its warps take the pieces of the listed
// blocks, 16 rows or a smaller block each, in turn.  Each warp runs alone: it
// looks up 32 pieces at a time (one per lane: list entry, table entry, rows
// covered), makes 16-row tiles of them (with a tile a block, 33 sequences of 101
// blocks of 8 rows, fp32, Hkv 8, D 64, took 47 us instead of 30), keeps a ring of
// tiles in flight with 16-byte cp.async copies to its own shared memory (rows
// that the query does not see arrive as zeros, so whatever they hold never
// enters a product), and holds its own running softmax state:
//   bf16: S^T = K Q^T with the tile's 16 tokens as M of mma m16n8k16 and the
//     heads as N; the weights go to the B operand of O^T += V^T P^T with one
//     movmatrix per 8 x 8.  An mma takes one type, that of V, and a bf16 weight
//     alone would be the largest error of the result (0.0022 of its norm
//     instead of 0.0017, which is the output's own rounding): each weight
//     enters as the next bf16 below it and the bf16 of what that leaves,
//     within 2^-16 of it together, in two products (83 us either way on 64
//     sequences x 2048 tokens).  The statistics and O stay in fp32.
//   int8: the same on fp16 mma over the exact codes, q scaled into fp16 by a
//     power of two.  V's scales are folded into the weights; the products of a
//     head are taken in units of a power of two in which the largest of them, as
//     weights stand now, is 2^2 to 2^15, and each enters as an fp16 and the fp16 of
//     what that leaves: within 2^-22 of it, or 2^-27 of the largest.  (One fp16
//     alone, in units of the largest V scale, lost all of a result to a row of next
//     to no weight whose scale was 2^30 that of the others.  64 sequences x 2048
//     tokens, 8 kv heads, D 128, with G 4 and 16: that one part 67.9 and 80.9 us,
//     two parts 68.7 and 89.3; two bf16 parts, which need no units, 71.4 and 97.3:
//     a code takes twice the instructions to bf16.)  With up to 4 heads a group the
//     second parts take the columns that the first leave empty: one mma, not two.
//     The rows of a tile are taken in the order that makes the byte-transposing V
//     load agree with movmatrix.
//   fp32: fp32 FMAs, two lanes per token for the scores, D / 32 output dims
//     per lane.
// At the end the warps' states (m, l, O) are merged by the log-sum-exp rule
// out of the shared memories of the whole cluster: no workspace, no second
// kernel.
#include <climits>
#include <cmath>
#include <type_traits>

#include "cluster.cuh"
#include "common.cuh"
#include "mma.cuh"
#include "span.cuh"

namespace pkv {
namespace {

constexpr int kTile = 16;       // rows of a tile
constexpr int kMaxWarps = 8;    // of a CTA
constexpr int kMaxCluster = 8;  // CTAs
constexpr int kMaxStates = 48;  // warps of a cluster (with 64, 16 us where 48 take 13)
constexpr int kStates = 64;     // room for them, two a lane in their merge
// One sequence under a window of 4096, 8 kv heads, D 128, G 4, bf16, by warps x CTAs: 8 x 6 11.5
// us, 4 x 12 10.0, 4 x 16 11.4; of 16384 24.7, 20.1, 21.1; of 65536 78.8, 62.2, 61.2.
constexpr int kWideCluster = 16;
constexpr int kLongWindow = 512;  // tiles
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

// int8: products of weights and V scales in units of O.  Units are chosen so that
// the largest is 2^6 to 2^7 of them, for exponents of it from kLeastTop to kMostTop, and
// again once it has moved by more than 2^kDrift or a scale passes kMostProduct:
// scales up to 2^8 times the largest product need no look at the products.
constexpr float kMostProduct = 32768.f;
constexpr int kDrift = 4, kLeastTop = -120, kMostTop = 127;

struct SparseParams {
  const char* k;
  const char* v;
  const char* q;
  char* out;
  const int32_t* bt;
  const int32_t* offs;
  const int32_t* tok_seq;
  const int32_t* tok_pos;
  const int32_t* sel;
  int* err;
  long long num_blocks;
  int batch, mb, bs, L, layer, row_bytes, scale_off, hq, hkv, G, K;
  int parts;      // pieces of a block (a power of two)
  int piece_bits; // log2 of the rows of a piece
  float qscale;   // scale * log2(e)
  // the window form: K is then the number of blocks that a query sees at most
  const int32_t* lens;
  int window, sink;
};

// ---- small helpers -----------------------------------------------------------

// Transpose of an 8 x 8 matrix of 16-bit elements held one row pair a lane.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// ---- staging -------------------------------------------------------------------

// One tile in a warp's ring: K rows, V rows, and for int8 pools their scales.
template <int MODE, int D>
struct Tile {
  static constexpr int kEs = MODE == PKV_F32 ? 4 : MODE == PKV_BF16 ? 2 : 1;
  static constexpr int kRow = D * kEs;              // bytes of one head of a row
  static constexpr int kChunks = kRow / 16;         // 16-byte chunks of it
  static constexpr int kHalf = kTile * kRow;        // K (or V) rows
  static constexpr int kScales = MODE == PKV_I8 ? 2 * kTile * 16 : 0;
  static constexpr int kBytes = 2 * kHalf + kScales;
  // Byte offset of chunk c of row r: chunks of a row are permuted so that the
  // 8 rows of an ldmatrix (and the 2 rows x 4 chunks of an LDS.128 phase of
  // the int8 K reads) fall in 8 different 16-byte columns.
  static __device__ __forceinline__ int at(int r, int c) {
    if constexpr (MODE == PKV_I8) {
      if constexpr (D == 64) return r * kRow + ((c ^ ((r >> 1) & 3)) << 4);
      return r * kRow + ((c ^ (((r & 1) << 2) | ((r >> 1) & 3))) << 4);
    }
    return r * kRow + ((c ^ (r & 7)) << 4);
  }

  // Start the copies of the tile's rows in `mask`; the others are filled with
  // zeros (no byte of them is read).  `row` of lane u: the token row of the first
  // row of piece u; a tile of one piece passes ONE.
  template <bool ONE>
  static __device__ __forceinline__ void load(const SparseParams& p, uint32_t dst, long long row,
                                              int g, uint32_t mask, int lane) {
    constexpr int RPI = 32 / (kChunks < 32 ? kChunks : 32);  // rows of one instruction
    const long long row0 = ONE ? row : __shfl_sync(kAll, row, 0);
    // bytes from row0 to row r (0 for a row that is not copied)
    auto bytes_to = [&](int r) -> long long {
      const bool live = mask >> r & 1;
      if constexpr (ONE) return live ? (long long)r * p.row_bytes : 0;
      const long long at_row =
          __shfl_sync(kAll, row, r >> p.piece_bits) + (r & ((1 << p.piece_bits) - 1));
      return live ? (at_row - row0) * p.row_bytes : 0;
    };
    const char* kb = p.k + row0 * p.row_bytes;
    const char* vb = p.v + row0 * p.row_bytes;
    const int c = lane % kChunks, r0 = lane / kChunks, col = g * kRow + c * 16;
#pragma unroll
    for (int i = 0; i < kTile / RPI; ++i) {
      const int r = i * RPI + r0;
      const long long off = bytes_to(r) + col;
      cp_async16(dst + at(r, c), kb + off, mask >> r & 1);
      cp_async16(dst + kHalf + at(r, c), vb + off, mask >> r & 1);
    }
    if constexpr (MODE == PKV_I8) {
      const int r = lane & 15;
      // the 16 bytes that hold the head's scale (rows are padded to 16)
      const char* src = (lane < 16 ? kb : vb) + bytes_to(r) + p.scale_off + (4 * g & ~15);
      cp_async16(dst + 2 * kHalf + lane * 16, src, mask >> r & 1);
    }
  }
};

// ---- consumers: the running state of one warp ------------------------------------

// Tensor-core state for bf16 and int8 pools.  HEADS 4 (int8): the heads stand twice
// among the 8 columns, and in the product with V the weights' first parts take
// columns 0-3 and what is left of them 4-7.
template <int MODE, int D, int HEADS>
struct MmaState {
  static constexpr bool kI8 = MODE == PKV_I8, kTwice = HEADS == 4;
  static constexpr int NT = (HEADS + 7) / 8;
  static constexpr int KS = D / 16;
  using Tl = Tile<MODE, D>;
  uint32_t qb[NT][KS][2];
  float o[NT][KS][4];
  float m[NT][2], l[NT][2];
  float qs[NT][2];  // factor of the scores of columns 2 qi, 2 qi + 1
  int so;           // int8: byte of the head's scale in its 16
  // int8: O of a column is held in units of 1 / unit.  drift: the logarithm of the
  // largest product, as weights stand now, over the power of two that the unit was
  // chosen for; widest: the largest unit of the lane's columns.
  float unit[NT][2], drift[NT][2], widest;
  static __device__ __forceinline__ float unit_of(int top) {
    return __uint_as_float((uint32_t)(133 - top) << 23);
  }

  // Off the usual path: units for the products `x` (weights times V scales) of a
  // tile, where the ones so far have drifted or may not hold them; a: factor of O.
  __device__ void choose_units(const float (&x)[NT][4], float (&a)[NT][2]) {
    widest = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mx = fmaxf(fabsf(x[nt][c]), fabsf(x[nt][c + 2]));
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
        const int old = 133 - (int)(__float_as_uint(unit[nt][c]) >> 23);
        // the largest of the tile's products and of those before
        const float most = fmaxf((float)((int)(__float_as_uint(mx) >> 23) - 127),
                                 (float)old + drift[nt][c]);
        const int top = min(kMostTop, max(kLeastTop, (int)floorf(most)));
        if (abs(top - old) > kDrift) {
          const int k = old - top;  // in two steps: 2^k may pass the range of fp32
          a[nt][c] *= __uint_as_float((uint32_t)(127 + k / 2) << 23);
          a[nt][c] *= __uint_as_float((uint32_t)(127 + (k - k / 2)) << 23);
          unit[nt][c] = unit_of(top);
          drift[nt][c] = fmaxf(most - (float)top, 0.f);
        } else {
          drift[nt][c] = most - (float)old;
        }
        widest = fmaxf(widest, unit[nt][c]);
      }
  }

  __device__ void init(const SparseParams& p, int t, int g, int lane) {
    const int gl = lane >> 2, qi = lane & 3;
    so = 4 * g & 15;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
      unit[nt][0] = unit[nt][1] = widest = unit_of(kLeastTop);
      drift[nt][0] = drift[nt][1] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nt][k][c] = 0.f;
      const int h = kTwice ? gl & 3 : nt * 8 + gl;
      const bool live = h < p.G;
      const char* src = p.q + ((long long)t * p.hq + g * p.G + (live ? h : 0)) * (D * 2);
      if constexpr (!kI8) {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qb[nt][k][i] = live ? *reinterpret_cast<const uint32_t*>(
                                      src + (k * 16 + i * 8 + qi * 2) * 2)
                                : 0u;
        qs[nt][0] = qs[nt][1] = p.qscale;
      } else {
        // dims i * 64 + qi * 16 .. + 15: the order of the K codes (scores())
        uint32_t w[KS / 4][8], mx = 0;
#pragma unroll
        for (int i = 0; i < KS / 4; ++i)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint4 r = live ? *reinterpret_cast<const uint4*>(src + (i * 64 + qi * 16) * 2 +
                                                                   16 * v)
                                 : make_uint4(0, 0, 0, 0);
            w[i][4 * v] = r.x; w[i][4 * v + 1] = r.y; w[i][4 * v + 2] = r.z; w[i][4 * v + 3] = r.w;
          }
#pragma unroll
        for (int i = 0; i < KS / 4; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mx = max(mx, max(w[i][k] & 0x7FFFu, (w[i][k] >> 16) & 0x7FFFu));
        mx = max(mx, __shfl_xor_sync(kAll, mx, 1));
        mx = max(mx, __shfl_xor_sync(kAll, mx, 2));
        // 2^e brings the absmax into [2^14, 2^15): fp16 holds every bf16
        // value down to 2^-28 of it exactly
        int e = 0;
        if (mx != 0) e = min(126, max(-126, 141 - (int)((mx >> 7) & 0xFF)));
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < KS / 4; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            qb[nt][i * 4 + k / 2][k & 1] =
                pack_f16x2(bf16_lo(w[i][k]) * up, bf16_hi(w[i][k]) * up);
        qs[nt][0] = p.qscale * __shfl_sync(kAll, down, 8 * qi);
        qs[nt][1] = p.qscale * __shfl_sync(kAll, down, 8 * qi + 4);
      }
    }
  }

  // One staged tile; the rows in `mask` are the ones the query sees.
  __device__ void step(uint32_t st, uint32_t mask, int lane) {
    const int gl = lane >> 2, qi = lane & 3;
    // the tokens of this lane's two score rows
    const int t0 = kI8 ? 4 * (gl >> 1) + (gl & 1) : gl, t1 = kI8 ? t0 + 2 : gl + 8;
    const bool in0 = mask >> t0 & 1, in1 = mask >> t1 & 1;
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[nt][c] = 0.f;
    if constexpr (!kI8) {
      const int r = (lane & 7) + ((lane >> 3) & 1) * 8, cc = lane >> 4;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[4];
        ldsm_x4(a, st + Tl::at(r, 2 * k + cc));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16<false>(s[nt], a[0], a[1], a[2], a[3], qb[nt][k][0], qb[nt][k][1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < KS / 4; ++i) {
        const uint4 x = lds128(st + Tl::at(t0, 4 * i + qi)), y = lds128(st + Tl::at(t1, 4 * i + qi));
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a0, a1, a2, a3;
          codes_to_f16(xw[j], a0, a2);
          codes_to_f16(yw[j], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16<true>(s[nt], a0, a1, a2, a3, qb[nt][i * 4 + j][0], qb[nt][i * 4 + j][1]);
        }
      }
    }
    float sk0 = 1.f, sk1 = 1.f, sv0 = 1.f, sv1 = 1.f;
    if constexpr (kI8) {
      const uint32_t sc = st + 2 * Tl::kHalf + so;
      sk0 = lds_f32(sc + t0 * 16);
      sk1 = lds_f32(sc + t1 * 16);
      sv0 = lds_f32(sc + (16 + t0) * 16);
      sv1 = lds_f32(sc + (16 + t1) * 16);
    }
    float a[NT][2];  // factor of O
    bool moved = false;
    [[maybe_unused]] bool choose = false;  // int8: units of O
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      s[nt][0] = in0 ? s[nt][0] * qs[nt][0] * sk0 : -INFINITY;
      s[nt][1] = in0 ? s[nt][1] * qs[nt][1] * sk0 : -INFINITY;
      s[nt][2] = in1 ? s[nt][2] * qs[nt][0] * sk1 : -INFINITY;
      s[nt][3] = in1 ? s[nt][3] * qs[nt][1] * sk1 : -INFINITY;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mx = fmaxf(s[nt][c], s[nt][c + 2]);
        float shrink = 1.f;
        a[nt][c] = 1.f;
        // the running maximum moves only where some lane passes it
        if (__any_sync(kAll, mx > m[nt][c])) {
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
          const float n = fmaxf(m[nt][c], mx);
          // nothing but -inf so far: there is nothing to rescale
          shrink = m[nt][c] == -INFINITY ? 0.f : exp2f(m[nt][c] - n);
          a[nt][c] = shrink;
          if constexpr (kI8) {
            if (m[nt][c] != -INFINITY && n > m[nt][c]) drift[nt][c] += m[nt][c] - n;
            choose |= drift[nt][c] < -kDrift;
          }
          m[nt][c] = n;
        }
        // scores of -inf carry no weight, even while they are all there is
        const float base = m[nt][c] == -INFINITY ? 0.f : m[nt][c];
        s[nt][c] = exp2f(s[nt][c] - base);
        s[nt][c + 2] = exp2f(s[nt][c + 2] - base);
        l[nt][c] = l[nt][c] * shrink + s[nt][c] + s[nt][c + 2];
        moved |= a[nt][c] != 1.f;
      }
    }
    if constexpr (kI8) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[nt][c] *= c < 2 ? sv0 : sv1;
      // (no weight is above 1)
      choose |= fmaxf(fabsf(sv0), fabsf(sv1)) * widest > kMostProduct;
      moved |= choose;
    }
    if (__any_sync(kAll, moved)) {
      if constexpr (kI8) {
        if (__any_sync(kAll, choose)) choose_units(s, a);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          o[nt][k][0] *= a[nt][0];
          o[nt][k][1] *= a[nt][1];
          o[nt][k][2] *= a[nt][0];
          o[nt][k][3] *= a[nt][1];
        }
    }
    uint32_t pb[NT][2];  // the first parts of the weights (times V scales),
    [[maybe_unused]] uint32_t rest[NT][2];  // and what is left of them
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t h[2], r[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = s[nt][2 * i], y = s[nt][2 * i + 1];
        if constexpr (kI8) {
          x *= unit[nt][0];
          y *= unit[nt][1];
          h[i] = pack_f16x2_finite(x, y);
          const float2 f = unpack_f16x2(h[i]);
          r[i] = pack_f16x2(x - f.x, y - f.y);
        } else {
          h[i] = below_bf16x2(x, y);
          r[i] = pack_bf16x2(x - bf16_lo(h[i]), y - bf16_hi(h[i]));
        }
        pb[nt][i] = movmatrix_t(kTwice && qi >= 2 ? r[i] : h[i]);
        if constexpr (!kTwice) rest[nt][i] = movmatrix_t(r[i]);
      }
    }
    const uint32_t sv = st + Tl::kHalf;
    if constexpr (!kI8) {
      const int r = (lane & 7) + (lane >> 4) * 8, cc = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t v[4];
        ldsm_x4_t(v, sv + Tl::at(r, 2 * k + cc));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16<false>(o[nt][k], v[0], v[1], v[2], v[3], pb[nt][0], pb[nt][1]);
          mma16<false>(o[nt][k], v[0], v[1], v[2], v[3], rest[nt][0], rest[nt][1]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < KS; k += 2) {  // (two at a time: products into one sum lie apart)
        uint32_t v[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t r0, r1;
          ldsm_b8_t(r0, r1, sv + Tl::at(lane & 15, k + u));
          codes_to_f16(r0, v[u][0], v[u][2]);
          codes_to_f16(r1, v[u][1], v[u][3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16<true>(o[nt][k + u], v[u][0], v[u][1], v[u][2], v[u][3], pb[nt][0], pb[nt][1]);
        }
        if constexpr (!kTwice) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16<true>(o[nt][k + u], v[u][0], v[u][1], v[u][2], v[u][3], rest[nt][0],
                          rest[nt][1]);
        }
      }
    }
  }

  // The state to shared memory: O as [head][D], then (m, l) of each head.
  __device__ void put(const SparseParams& p, uint32_t acc, uint32_t ml, int lane) {
    const int gl = lane >> 2, qi = lane & 3;
    if constexpr (kTwice) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[0][k][c] += __shfl_xor_sync(kAll, o[0][k][c], 2);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = l[nt][c];
        x += __shfl_xor_sync(kAll, x, 4);
        x += __shfl_xor_sync(kAll, x, 8);
        x += __shfl_xor_sync(kAll, x, 16);
        const int h = nt * 8 + 2 * qi + c;
        // int8: back to the units of V
        const float back = kI8 ? __uint_as_float((254u << 23) - __float_as_uint(unit[nt][c])) : 1.f;
        if (h < p.G) {
          if (gl == 0) {
            sts_f32(ml + h * 8, m[nt][c]);
            sts_f32(ml + h * 8 + 4, x);
          }
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            sts_f32(acc + (h * D + k * 16 + gl) * 4, o[nt][k][c] * back);
            sts_f32(acc + (h * D + k * 16 + gl + 8) * 4, o[nt][k][c + 2] * back);
          }
        }
      }
  }
};

// fp32 state: GP heads (G rounded up), q and the weights in shared memory.
template <int D, int GP>
struct FmaState {
  using Tl = Tile<PKV_F32, D>;
  static constexpr int PD = D / 32;  // output dims of a lane
  float o[GP][PD], m[GP], l[GP];     // l: this lane's token's share
  uint32_t sq, sp;

  static constexpr int kExtra = (GP * D + kTile * GP) * 4;  // q, weights

  __device__ void init(const SparseParams& p, int t, int g, int lane, uint32_t extra) {
    sq = extra;
    sp = extra + GP * D * 4;
#pragma unroll
    for (int h = 0; h < GP; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int e = 0; e < PD; ++e) o[h][e] = 0.f;
    }
    const char* src = p.q + ((long long)t * p.hq + g * p.G) * (D * 4) + lane * 16;
    uint4 x[GP * D / 128];
#pragma unroll
    for (int i = 0; i < GP * D / 128; ++i)
      x[i] = i * 128 + lane * 4 < p.G * D ? ld_stream(src + i * 512) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < GP * D / 128; ++i) {
      const uint32_t at = sq + i * 512 + lane * 16;
      sts_f32(at, __uint_as_float(x[i].x) * p.qscale);
      sts_f32(at + 4, __uint_as_float(x[i].y) * p.qscale);
      sts_f32(at + 8, __uint_as_float(x[i].z) * p.qscale);
      sts_f32(at + 12, __uint_as_float(x[i].w) * p.qscale);
    }
    __syncwarp();
  }

  __device__ void step(uint32_t st, uint32_t mask, int lane) {
    const int tok = lane & 15, side = lane >> 4;  // two lanes a token, half the dims each
    const bool in = mask >> tok & 1;
#pragma unroll
    for (int h0 = 0; h0 < GP; h0 += 4) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const int ch = side * (D / 8) + c;
        const uint4 kr = lds128(st + Tl::at(tok, ch));
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint4 qr = lds128(sq + ((h0 + h) * D + ch * 4) * 4);
          s[h] = fmaf(__uint_as_float(qr.x), __uint_as_float(kr.x), s[h]);
          s[h] = fmaf(__uint_as_float(qr.y), __uint_as_float(kr.y), s[h]);
          s[h] = fmaf(__uint_as_float(qr.z), __uint_as_float(kr.z), s[h]);
          s[h] = fmaf(__uint_as_float(qr.w), __uint_as_float(kr.w), s[h]);
        }
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float x = s[h] + __shfl_xor_sync(kAll, s[h], 16);
        x = in ? x : -INFINITY;
        float a = 1.f;
        if (__any_sync(kAll, x > m[h0 + h])) {
          float mx = x;
#pragma unroll
          for (int b = 8; b; b >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, b));
          const float n = fmaxf(m[h0 + h], mx);
          a = m[h0 + h] == -INFINITY ? 0.f : exp2f(m[h0 + h] - n);
          m[h0 + h] = n;
#pragma unroll
          for (int e = 0; e < PD; ++e) o[h0 + h][e] *= a;
        }
        const float w = exp2f(x - (m[h0 + h] == -INFINITY ? 0.f : m[h0 + h]));
        l[h0 + h] = l[h0 + h] * a + w;
        if (side == 0) sts_f32(sp + (tok * GP + h0 + h) * 4, w);
      }
    }
    __syncwarp();
    const uint32_t sv = st + Tl::kHalf;
#pragma unroll 4
    for (int t = 0; t < kTile; ++t) {
      float v[PD];
      const int byte = lane * PD * 4;
      const uint32_t va = sv + Tl::at(t, byte >> 4) + (byte & 15);
      if constexpr (PD == 4) {
        const uint4 r = lds128(va);
        v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
      } else {
#pragma unroll
        for (int e = 0; e < PD; ++e) v[e] = lds_f32(va + 4 * e);
      }
#pragma unroll
      for (int h0 = 0; h0 < GP; h0 += 4) {
        const uint4 w = lds128(sp + (t * GP + h0) * 4);
        const float wf[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                             __uint_as_float(w.w)};
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
          for (int e = 0; e < PD; ++e) o[h0 + h][e] = fmaf(wf[h], v[e], o[h0 + h][e]);
      }
    }
    __syncwarp();
  }

  __device__ void put(const SparseParams& p, uint32_t acc, uint32_t ml, int lane) {
#pragma unroll
    for (int h = 0; h < GP; ++h) {
      float x = l[h];
#pragma unroll
      for (int b = 8; b; b >>= 1) x += __shfl_xor_sync(kAll, x, b);
      if (h < p.G) {
        if (lane == 0) {
          sts_f32(ml + h * 8, m[h]);
          sts_f32(ml + h * 8 + 4, x);
        }
#pragma unroll
        for (int e = 0; e < PD; ++e) sts_f32(acc + (h * D + lane * PD + e) * 4, o[h][e]);
      }
    }
  }
};

// ---- the kernel -------------------------------------------------------------------

// HEADS: heads the state holds, G rounded up (bf16: 8 or 16, the others 4 too).
template <int MODE, int D, int HEADS>
struct Layout {
  using Tl = Tile<MODE, D>;
  // Tiles of a warp's ring: three; two where a tile is large (fp32) or its work long
  // beside its bytes (int8, D 128).  Times over those of the best count from 2 to 8 of
  // each of 11 batches (1 to 128 sequences, 40 to 300 blocks of 16; geometric means):
  // bf16, D 64, G 2 to 16: with 3 1.02-1.06, with 2 1.07-1.10, 4 1.03-1.09, 5 1.05-1.14;
  // int8, D 64, G 4 to 16: 3 1.02-1.04, 2 1.03-1.04, 4 1.04-1.06, 8 1.14-1.19; int8,
  // D 128, G 12 and 16: 2 1.01, 3 1.01-1.02, 5 1.04.  64 sequences x 2048 tokens, G 4,
  // D 128: bf16 with 3 81.8 us, 2 82.5, 4 88.3; int8 2 64.4, 3 70.0, 5 67.5; fp32, 32
  // sequences, 2 84.9, 3 90.6.
  static constexpr int kStages = MODE == PKV_F32 || (MODE == PKV_I8 && D == 128) ? 2 : 3;
  static constexpr int kRing = kStages * Tl::kBytes;
  static constexpr int kState = HEADS * D * 4 + HEADS * 8;  // of the merge; over the ring
  static constexpr int kBody = (kRing > kState ? kRing : kState);
  static constexpr int kExtra = MODE == PKV_F32 ? FmaState<D, HEADS>::kExtra : 0;
  static constexpr int kWarp = (kBody + kExtra + 127) / 128 * 128;
  static constexpr int kStatic = (HEADS + 1) * kStates * 4;  // the merge's weights, addresses
  static constexpr int kFit = (227 * 1024 - kStatic) / kWarp;
  static constexpr int kLimit = MODE == PKV_F32 && HEADS > 8 ? 4 : kMaxWarps;  // (4 fill the FMAs)
  static constexpr int kWarps = kFit < kLimit ? kFit : kLimit;  // of a CTA at most
};

// WINDOW: the query of row t is the last token of sequence t, and its blocks are no list
// but those with one of the first `sink` or the last `window` tokens.
template <int MODE, int D, int HEADS, bool WINDOW>
__global__ void __launch_bounds__(Layout<MODE, D, HEADS>::kWarps * 32)
    sparse_decode_kernel(const SparseParams p) {
  using Tl = Tile<MODE, D>;
  using Lay = Layout<MODE, D, HEADS>;
  constexpr int NST = Lay::kStages;
  const int W = blockDim.x >> 5;  // warps of a CTA
  extern __shared__ __align__(128) unsigned char smem[];
  griddep_wait();
  griddep_launch_dependents();
  uint32_t S;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const uint32_t rank = cluster_rank();
  const int row = blockIdx.x / S;
  const int t = row / p.hkv, g = row - t * p.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // The chain of loads before the first row arrives is list, sequence and
  // position; offset and table entry; row: a batch's list entries are loaded one
  // batch ahead, the first ones here.
  const int32_t* list = WINDOW ? nullptr : p.sel + (long long)row * p.K;
  int all_pieces = p.K * p.parts;
  // window form: the first `heads` listed blocks are the table's first, the others follow
  // from block `tail` on; table positions [hide_lo, hide_hi) are not seen
  [[maybe_unused]] int heads = 0, tail = 0, hide_lo = 0, hide_hi = 0;
  const int part_bits = 31 - __clz(p.parts);
  const int stride = (int)S * W;
  int next = (int)rank * W + warp;  // first piece of the batch to come
  auto listed = [&](long long ts) {
    if (ts >= all_pieces) return -1;
    const int u = (int)(ts >> part_bits);
    if constexpr (WINDOW) return u < heads ? u : tail + (u - heads);
    return ld_volatile(list + u);
  };
  int ahead = WINDOW ? -1 : listed(next + (long long)lane * stride);
  const int seq = WINDOW ? t : ld_volatile(p.tok_seq + t);
  const int pos = WINDOW ? ld_volatile(p.lens + t) - 1 : ld_volatile(p.tok_pos + t);
  if (seq < 0) return;  // padding: the whole cluster leaves, nothing is written
  int off = 0, end = 0;  // table positions [off, end) are seen
  if (seq >= p.batch) {
    if (rank == 0 && tid == 0) set_error(p.err, kErrIndex);
  } else {
    off = p.offs ? p.offs[seq] : 0;
    if (off < 0 || off >= p.bs || pos < (WINDOW ? -1 : 0) ||
        (long long)off + pos >= (long long)p.mb * p.bs) {
      if (rank == 0 && tid == 0) set_error(p.err, kErrCapacity);
    } else if (!WINDOW || pos >= 0) {
      end = off + pos + 1;
    }
  }
  if constexpr (WINDOW) {
    if (end > 0) {
      const int bs_bits = 31 - __clz(p.bs);
      hide_lo = min(off + p.sink, end);
      hide_hi = max(off, end - p.window);
      tail = hide_hi >> bs_bits;
      const int last_head = min(hide_lo, hide_hi) - 1;
      heads = last_head >= off ? min((last_head >> bs_bits) + 1, tail) : 0;
      all_pieces = (heads + ((end - 1) >> bs_bits) - tail + 1) * p.parts;
      ahead = listed(next + (long long)lane * stride);
    }
  }
  const int pieces = end > 0 ? all_pieces : 0;  // a bad token sees nothing: zeros

  const uint32_t base = smem_addr(smem);
  const uint32_t ring = base + warp * Lay::kWarp;

  // ---- lookup: 32 pieces a time, one per lane ----
  const int32_t* table = p.bt + (long long)(end > 0 ? seq : 0) * p.mb;
  const int rows_piece = 1 << p.piece_bits;
  long long my_row = 0;
  uint32_t my_mask = 0;
  unsigned todo = 0;
  auto lookup = [&]() {
    // stops at the last batch or at one that has something to do
    while (todo == 0 && next < pieces) {
      const long long ts = next + (long long)lane * stride;
      const int j = ahead;
      ahead = listed(ts + 32ll * stride);
      int lo = 0, hi = 0;
      if (j >= p.mb) set_error(p.err, kErrIndex);
      uint32_t hidden = 0;
      if (j >= 0 && j < p.mb) {
        const int r0 = (int)(ts & (p.parts - 1)) * kTile;
        const int p0 = j * p.bs + r0;
        lo = max(0, off - p0);
        hi = min(rows_piece, end - p0);
        if constexpr (WINDOW) {
          const int a = max(0, hide_lo - p0), b = min(rows_piece, hide_hi - p0);
          if (a < b) hidden = (1u << b) - (1u << a);
          // a block without a token that is seen is not looked up
          if (lo >= hi || (((1u << hi) - (1u << lo)) & ~hidden) == 0) lo = hi = 0;
        }
        const int blk = WINDOW && lo >= hi ? 0 : ld_volatile(table + j);
        if (blk >= 0 && blk < p.num_blocks) {
          my_row = ((long long)blk * p.L + p.layer) * p.bs + r0;
        } else if (lo < hi) {
          set_error(p.err, kErrIndex);
          hi = 0;
        }
      }
      my_mask = lo < hi ? ((1u << hi) - (1u << lo)) & ~hidden : 0u;
      todo = __ballot_sync(kAll, lo < hi);
      next = pieces - next <= 32 * stride ? pieces : next + 32 * stride;
    }
  };
  uint32_t masks = 0;  // lane s: the rows of the tile in stage s
  auto issue = [&](int stage) {
    lookup();
    uint32_t mask = 0;
    if (todo) {
      const uint32_t dst = ring + stage * Tl::kBytes;
      int src = __ffs(todo) - 1;
      todo &= todo - 1;
      long long r = __shfl_sync(kAll, my_row, src);
      mask = __shfl_sync(kAll, my_mask, src);
      if (rows_piece == kTile) {
        Tl::template load<true>(p, dst, r, g, mask, lane);
      } else {
        for (int u = 1; u < kTile >> p.piece_bits; ++u) {
          lookup();
          if (todo == 0) break;
          src = __ffs(todo) - 1;
          todo &= todo - 1;
          const long long x = __shfl_sync(kAll, my_row, src);
          mask |= __shfl_sync(kAll, my_mask, src) << (u << p.piece_bits);
          if (lane >= u) r = x;
        }
        Tl::template load<false>(p, dst, r, g, mask, lane);
      }
    }
    if (lane == stage) masks = mask;
    cp_commit();
  };

  // The query: bf16 fragments are plain loads and go ahead of the tiles; the
  // others compute on it, while the first tiles arrive.
  std::conditional_t<MODE == PKV_F32, FmaState<D, HEADS>,
                     MmaState<MODE == PKV_F32 ? PKV_BF16 : MODE, D, HEADS>>
      state;
  if constexpr (MODE == PKV_BF16) state.init(p, t, g, lane);
#pragma unroll 1
  for (int s = 0; s < NST - 1; ++s) issue(s);
  if constexpr (MODE == PKV_F32) state.init(p, t, g, lane, ring + Lay::kBody);
  if constexpr (MODE == PKV_I8) state.init(p, t, g, lane);
  int stage = 0;
#pragma unroll 1
  while (true) {
    cp_wait<NST - 2>();
    __syncwarp();
    const uint32_t mask = __shfl_sync(kAll, masks, stage);
    if (mask == 0) break;
    issue(stage == 0 ? NST - 1 : stage - 1);
    state.step(ring + stage * Tl::kBytes, mask, lane);
    if (++stage == NST) stage = 0;
  }
  cp_wait<0>();
  __syncwarp();

  // ---- merge of the cluster's warps ----
  const uint32_t acc = ring, ml = ring + HEADS * D * 4;
  state.put(p, acc, ml, lane);
  if (S > 1)
    cluster_sync();
  else
    __syncthreads();
  // weights of the S * W states of each head
  __shared__ float weight[HEADS][kStates];
  __shared__ uint32_t state_at[kStates];
  const int states = (int)S * W;
  uint32_t at[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int j = min(lane + 32 * u, states - 1);
    at[u] = cluster_map(base + (j % W) * Lay::kWarp, j / W);
    if (warp == 0) state_at[lane + 32 * u] = at[u];
  }
  for (int h = warp; h < p.G; h += W) {
    float m[2] = {-INFINITY, -INFINITY}, f[2], M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = lane + 32 * u;
      f[u] = 0.f;
      if (j < states) {
        m[u] = ld_cluster_f32(at[u] + HEADS * D * 4 + h * 8);
        f[u] = ld_cluster_f32(at[u] + HEADS * D * 4 + h * 8 + 4);
      }
      M = fmaxf(M, m[u]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // a state at -inf saw nothing, or only NaN: its l and O are 0, or NaN
      const float l = f[u];
      f[u] = m[u] == -INFINITY ? 1.f : exp2f(m[u] - M);
      sum += f[u] * l;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
#pragma unroll
    for (int u = 0; u < 2; ++u)  // no weight at all: zeros
      weight[h][lane + 32 * u] = sum == 0.f ? 0.f : f[u] / sum;
  }
  __syncthreads();
  const int pairs = p.G * (D / 2);
  for (int i = (int)(rank * blockDim.x) + tid; i < pairs; i += (int)(S * blockDim.x)) {
    const int h = i / (D / 2), d = (i % (D / 2)) * 2;
    float x = 0.f, y = 0.f;
#pragma unroll 8
    for (int j = 0; j < states; ++j) {
      float u, v;
      asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];"
                   : "=f"(u), "=f"(v)
                   : "r"(state_at[j] + (h * D + d) * 4));
      x += weight[h][j] * u;
      y += weight[h][j] * v;
    }
    const long long dst = ((long long)t * p.hq + g * p.G + h) * D + d;
    if constexpr (MODE == PKV_F32) {
      *reinterpret_cast<float2*>(p.out + dst * 4) = make_float2(x, y);
    } else {
      *reinterpret_cast<uint32_t*>(p.out + dst * 2) = pack_bf16x2(x, y);
    }
  }
  if (S > 1) cluster_sync();  // no CTA leaves while another may still read its states
}

// Warps W of a CTA and CTAs S of a cluster.  All that the device holds at once
// should have work, and the rows should fill whole rounds of it.  A warp's time
// for a tile grows with the L warps on its SM, about as 12 + L; a round costs it
// half a tile more, and a cluster 2 (1 beside the longer fp32 tiles) and a quarter
// for each of its CTAs.  The pair with the least
//     rounds * (tiles of a warp + 1/2 + 2 + S / 4) * (12 + L)
// is taken, clusters where one round is enough and with two tiles or more a warp.
// Of 50 cases of all types timed with every pair, it is within 5 % of the best in
// 45 and within 14 % in 48; 80 rows of 100 blocks, D 64, G 16, take 18 % (int8) and 27 %
// (bf16) more than with 6 x 3.  R rows of K blocks of 16, D 128, G 4, by W x S:
// fp32, R 264, K 60 3 x 1 45.6 us, 4 x 1 52.1, 2 x 1 57.7; R 160, K 100 1 x 5 48.1,
// 3 x 1 64.1, 4 x 1 76.9; bf16, R 512, K 128 2 x 1 83.0, 4 x 1 84.5, 8 x 1 92.2,
// 3 x 1 107; R 40, K 100 8 x 3 10.6, 4 x 3 11.4, 3 x 7 12.5; R 16, K 300 8 x 6 14.4,
// 4 x 8 14.8.
template <int MODE, int D, int HEADS, bool WINDOW>
cudaError_t launch_sparse_heads(const SparseParams& p, unsigned rows, int dev, int sms,
                                cudaStream_t s) {
  using Lay = Layout<MODE, D, HEADS>;
  // windows: clusters of up to 16 CTAs, and up to 64 states where these are long
  constexpr int kMost = WINDOW ? kWideCluster : kMaxCluster;
  static std::atomic<int> allowed[kDevices], known[kDevices][kMaxWarps + 1][kMost + 1];
  const auto kern = sparse_decode_kernel<MODE, D, HEADS, WINDOW>;
  cudaError_t e = allow_shared(kern, (size_t)Lay::kWarps * Lay::kWarp, allowed[dev]);
  if (e != cudaSuccess) return e;
  if constexpr (WINDOW) {
    static std::atomic<int> wide[kDevices];
    if ((e = allow_wide_clusters(kern, wide[dev])) != cudaSuccess) return e;
  }
  const long long tiles = ((long long)p.K * p.parts << p.piece_bits) / kTile;
  int warps = 1, ctas = 1;
  long long least = LLONG_MAX;
  constexpr bool kF32 = MODE == PKV_F32;
  for (const int W : {8, 6, 4, 3, 2, 1}) {
    // (beside the tensor cores' short tiles 6 warps and 1, and clusters below 4, gain nothing)
    if (W > Lay::kWarps || (!kF32 && (W == 6 || W == 1))) continue;
    const int most_states = WINDOW && tiles >= kLongWindow ? kStates : kMaxStates;
    for (int S = 1; S <= kMost && W * S <= most_states; ++S) {
      if (S > 1 && (tiles < 2 * W * S || (!kF32 && W < 4))) break;
      int fit = 0;
      e = clusters_held(kern, W * 32, (size_t)W * Lay::kWarp, (unsigned)S, known[dev][W][S], &fit);
      if (e != cudaSuccess) return e;
      if (fit < 1 || (S > 1 && rows > (unsigned)fit)) break;
      const long long rounds = (rows + (long long)fit - 1) / fit;
      const long long held = rounds > 1 ? fit : (long long)rows * S;
      const long long L = W * ((held + sms - 1) / sms);
      const long long each = (tiles + W * S - 1) / (W * S);  // tiles of a warp
      const long long more = S > 1 ? (kF32 ? 4 : 8) + S : 0;
      const long long cost = rounds * (4 * each + 2 + more) * (12 + L);
      if (cost < least) {
        least = cost;
        warps = W;
        ctas = S;
      }
    }
  }
  return launch_clusters(kern, dim3(rows * (unsigned)ctas), dim3(warps * 32),
                         (size_t)warps * Lay::kWarp, (unsigned)ctas, s, p);
}

template <int MODE, int D, bool WINDOW>
cudaError_t launch_sparse_d(const SparseParams& p, unsigned rows, int dev, int sms,
                            cudaStream_t s) {
  if constexpr (MODE != PKV_BF16) {
    if (p.G <= 4) return launch_sparse_heads<MODE, D, 4, WINDOW>(p, rows, dev, sms, s);
  }
  if (p.G <= 8) return launch_sparse_heads<MODE, D, 8, WINDOW>(p, rows, dev, sms, s);
  return launch_sparse_heads<MODE, D, 16, WINDOW>(p, rows, dev, sms, s);
}

template <bool WINDOW>
cudaError_t launch_sparse(const PoolView& v, const SparseParams& p, unsigned rows, int dev, int sms,
                          cudaStream_t s) {
  const bool d64 = v.head_dim == 64;
  if (v.quant)
    return d64 ? launch_sparse_d<PKV_I8, 64, WINDOW>(p, rows, dev, sms, s)
               : launch_sparse_d<PKV_I8, 128, WINDOW>(p, rows, dev, sms, s);
  if (v.io_size == 2)
    return d64 ? launch_sparse_d<PKV_BF16, 64, WINDOW>(p, rows, dev, sms, s)
               : launch_sparse_d<PKV_BF16, 128, WINDOW>(p, rows, dev, sms, s);
  return d64 ? launch_sparse_d<PKV_F32, 64, WINDOW>(p, rows, dev, sms, s)
             : launch_sparse_d<PKV_F32, 128, WINDOW>(p, rows, dev, sms, s);
}

// The parameters that the two calls share.
SparseParams sparse_params(const PoolView& v, int layer, const void* q, int num_q_heads,
                           float scale, const int32_t* bt, int mb, const int32_t* offs, int batch,
                           void* out, int* err) {
  SparseParams p = {};
  p.k = v.k;
  p.v = v.v;
  p.q = static_cast<const char*>(q);
  p.out = static_cast<char*>(out);
  p.bt = bt;
  p.offs = offs;
  p.err = err;
  p.num_blocks = v.num_blocks;
  p.batch = batch;
  p.mb = mb;
  p.bs = v.block_size;
  p.L = v.num_layers;
  p.layer = layer;
  p.row_bytes = v.row_bytes;
  p.scale_off = v.scale_off;
  p.hq = num_q_heads;
  p.hkv = v.num_kv_heads;
  p.G = num_q_heads / v.num_kv_heads;
  p.parts = v.block_size > kTile ? v.block_size / kTile : 1;
  while (p.piece_bits < 4 && 1 << p.piece_bits < v.block_size) ++p.piece_bits;
  p.qscale = scale * kLog2e;
  return p;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_decode_attention_sparse(
    const pkv_pool* pool, int32_t layer, const void* q, int32_t num_q_heads, float scale,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* offsets, int32_t batch,
    const int32_t* token_seq, const int32_t* token_pos, int32_t num_tokens,
    const int32_t* selected, int32_t num_selected, void* out, cudaStream_t stream) {
  pkv::PoolView v;
  int st = pkv::pool_view(pool, true, &v);
  if (st != PKV_OK) return (pkv_status)st;
  if (layer < 0 || layer >= v.num_layers || batch < 0 || num_tokens < 0 || num_q_heads <= 0 ||
      num_selected < 0 || num_q_heads % v.num_kv_heads != 0 || !std::isfinite(scale))
    return PKV_ERR_INVALID_ARG;
  const int G = num_q_heads / v.num_kv_heads;
  if ((v.head_dim != 64 && v.head_dim != 128) || G > 16) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!q || !out || !token_seq || !token_pos || (num_selected > 0 && !selected) ||
      (batch > 0 && (!block_tables || max_blocks_per_seq <= 0)))
    return PKV_ERR_INVALID_ARG;
  if (!pkv::aligned(q, 16) || !pkv::aligned(out, 16) || !pkv::aligned(block_tables, 4) ||
      !pkv::aligned(offsets, 4) || !pkv::aligned(token_seq, 4) || !pkv::aligned(token_pos, 4) ||
      !pkv::aligned(selected, 4))
    return PKV_ERR_INVALID_ARG;
  const int mb = batch > 0 ? max_blocks_per_seq : 1;
  const int parts = v.block_size > pkv::kTile ? v.block_size / pkv::kTile : 1;
  const int64_t rows = (int64_t)num_tokens * v.num_kv_heads;
  const int64_t pieces = (int64_t)num_selected * parts;
  // table positions and pieces are 32-bit in the kernel
  if ((int64_t)mb * v.block_size > INT32_MAX || pieces > (1 << 30) ||
      rows > INT32_MAX / 8)
    return PKV_ERR_UNSUPPORTED;
  int optin, grid, validate, sms, dev;
  int* err;
  if ((st = pkv::device_facts(&optin, &err, &grid, &validate)) != PKV_OK) return (pkv_status)st;
  if ((st = pkv::device_sm_count(&sms, &dev)) != PKV_OK) return (pkv_status)st;
  if (validate) {
    if ((st = pkv::clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
    if ((st = pkv::launch_status(pkv::launch_validate_tokens(
             v, block_tables, mb, offsets, batch, token_seq, token_pos, num_tokens, err,
             stream))) != PKV_OK)
      return (pkv_status)st;
    if ((st = pkv::read_and_clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
  }
  pkv::SparseParams p = pkv::sparse_params(v, layer, q, num_q_heads, scale, block_tables, mb, offsets,
                                           batch, out, err);
  p.tok_seq = token_seq;
  p.tok_pos = token_pos;
  p.sel = selected;
  p.K = num_selected;
  const cudaError_t e = pkv::launch_sparse<false>(v, p, (unsigned)rows, dev, sms, stream);
  if ((st = pkv::launch_status(e)) != PKV_OK) return (pkv_status)st;
  return validate ? (pkv_status)pkv::read_and_clear_error_word(err, stream) : PKV_OK;
}

extern "C" pkv_status pkv_decode_attention_window(
    const pkv_pool* pool, int32_t layer, const void* q, int32_t num_q_heads, float scale,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
    const int32_t* offsets, int32_t batch, int32_t window, int32_t sink, void* out,
    cudaStream_t stream) {
  pkv::PoolView v;
  int st = pkv::pool_view(pool, true, &v);
  if (st != PKV_OK) return (pkv_status)st;
  if (layer < 0 || layer >= v.num_layers || batch < 0 || num_q_heads <= 0 || window < 1 ||
      sink < 0 || num_q_heads % v.num_kv_heads != 0 || !std::isfinite(scale))
    return PKV_ERR_INVALID_ARG;
  if ((v.head_dim != 64 && v.head_dim != 128) || num_q_heads / v.num_kv_heads > 16)
    return PKV_ERR_UNSUPPORTED;
  if (batch == 0) return PKV_OK;
  if (!q || !out || !block_tables || !seq_lens || max_blocks_per_seq <= 0)
    return PKV_ERR_INVALID_ARG;
  if (!pkv::aligned(q, 16) || !pkv::aligned(out, 16) || !pkv::aligned(block_tables, 4) ||
      !pkv::aligned(seq_lens, 4) || !pkv::aligned(offsets, 4))
    return PKV_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)batch * v.num_kv_heads;
  if ((int64_t)max_blocks_per_seq * v.block_size > pkv::kMaxPositions || rows > INT32_MAX / 8)
    return PKV_ERR_UNSUPPORTED;
  int optin, grid, validate, sms, dev;
  int* err;
  if ((st = pkv::device_facts(&optin, &err, &grid, &validate)) != PKV_OK) return (pkv_status)st;
  if ((st = pkv::device_sm_count(&sms, &dev)) != PKV_OK) return (pkv_status)st;
  pkv::SparseParams p = pkv::sparse_params(v, layer, q, num_q_heads, scale, block_tables,
                                           max_blocks_per_seq, offsets, batch, out, err);
  p.lens = seq_lens;
  p.window = window;
  p.sink = (int)(sink < pkv::kMaxPositions ? sink : pkv::kMaxPositions);
  if (validate) {
    pkv::SpanParams sp = {};
    sp.lens = seq_lens;
    sp.offs = offsets;
    sp.total_q = batch;
    sp.batch = batch;
    sp.mb = max_blocks_per_seq;
    sp.bs = v.block_size;
    sp.max_q_len = 1;
    sp.window = window;
    sp.sink = p.sink;
    if ((st = pkv::clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
    if ((st = pkv::launch_status(pkv::launch_validate_spans(sp, nullptr, nullptr, 0, block_tables,
                                                            v.num_blocks, err, stream))) != PKV_OK)
      return (pkv_status)st;
    if ((st = pkv::read_and_clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
  }
  // the blocks that a query sees at most: those of the first tokens, from any row of a block
  // on, and those of the window
  const int64_t bs = v.block_size;
  const int64_t most = (sink > 0 ? (bs - 1 + p.sink + bs - 1) / bs : 0) + (window + bs - 2) / bs + 1;
  p.K = (int)(most < max_blocks_per_seq ? most : max_blocks_per_seq);
  const cudaError_t e = pkv::launch_sparse<true>(v, p, (unsigned)rows, dev, sms, stream);
  if ((st = pkv::launch_status(e)) != PKV_OK) return (pkv_status)st;
  return validate ? (pkv_status)pkv::read_and_clear_error_word(err, stream) : PKV_OK;
}
