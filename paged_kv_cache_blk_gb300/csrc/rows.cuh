// Attention of several query rows a kv head over one stream of its keys, on mma.sync:
// the general form of pkv_decode_attention_tree and pkv_prefill_attention_window, for
// every pool type, head_dim 64 and 128, any group of heads and block size (prefill.cu
// holds the tcgen05 form for bf16 pools of head_dim 128).
//
// What is computed.  The rows of a unit are (new token, query head of kv head g) pairs
// of one sequence, M = 16 WR of them (WR 1, 2 or 4).  Softmax attention over the keys
// that each row sees (span.cuh: a window, first tokens, a mask among the new tokens), K
// and V read in place through the block table.
//
// How.  A CTA of 4 warps streams the unit's tiles of KT keys through a ring of cp.async
// stages; rows that no query of the unit sees arrive as zeros, and are not read.  WR
// warps share out the rows and WK = 4 / WR the keys of each tile, so few rows cost few
// products (16 rows: every warp takes a quarter of the keys).  Each warp holds Q in
// registers and a running softmax (maximum, sum, O) of its 16 rows over its keys; the WK
// states of a row are merged in shared memory at the end.
//   bf16: S = Q K^T and O += P V on mma m16n8k16.  A weight enters P V as two bf16 parts,
//     within 2^-16 of it together (one part alone would be the largest error of the result).
//   int8: the same: codes are whole numbers up to 127, exact in bf16, K's scales are
//     factors of the scores and V's of the weights.  The tile's keys are taken in the
//     order that makes the byte-transposing V load agree with the scores' registers.
//   fp32: mma m16n8k8 on tf32 in three products: x = hi + lo, each the nearest tf32, and
//     x y ~ hi hi + hi lo + lo hi, within 2^-21 of it.  The tensor cores add with
//     truncation, so the small products come first, and O is not their accumulator: each
//     tile's P V is summed from zero and added to O with rounding.
#pragma once

#include <climits>
#include <cmath>

#include "cluster.cuh"
#include "common.cuh"
#include "mma.cuh"
#include "repair.cuh"
#include "span.cuh"

namespace pkv {

struct RowsParams {
  PlanParams plan;
  const char* k;
  const char* v;
  const char* q;
  char* out;
  const int32_t* bt;
  const int32_t* q_pos;          // tree: positions of the queries, or NULL
  const unsigned long long* mask;  // tree: [total_q, words], or NULL (each token sees those before it)
  int words;
  int* err;
  float* part;  // states of split units
  long long num_blocks;
  int L, layer, row_bytes, scale_off, hq, bs_bits;
  Repair repair;
  int units_max;  // prefill: units of one kv head of the longest sequence
  long long keys_most;  // prefill: keys that a unit's rows see at most
  float qscale;   // scale * log2(e)
};

constexpr int kRowsWarps = 4;
constexpr int kRowsMaxCluster = 8;
constexpr int kRowsThreads = kRowsWarps * 32;

namespace {

constexpr unsigned kAllLanes = 0xffffffffu;

__device__ __forceinline__ uint32_t tf32_of(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = tf32_of(x);
  lo = tf32_of(x - __uint_as_float(hi));
}
// d += a b: 16 x 8 x 8
__device__ __forceinline__ void mma8_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four codes (bytes c + 128) to bf16 pairs.  The low 7 bits of a byte behind 0x43 are
// 128 + them; the byte's top bit says whether 128 or 256 is to be taken off.
__device__ __forceinline__ uint32_t codes_pair_bf16(uint32_t spread) {
  const uint32_t x = spread & 0xFF7FFF7Fu, y = (~spread & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                   *reinterpret_cast<const __nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  uint32_t a, b;
  asm("prmt.b32 %0, %1, 0x43434343, 0x4140;" : "=r"(a) : "r"(w));
  asm("prmt.b32 %0, %1, 0x43434343, 0x4342;" : "=r"(b) : "r"(w));
  lo = codes_pair_bf16(a);
  hi = codes_pair_bf16(b);
}

template <int MODE, int D>
struct RowsTile {
  static constexpr int kEs = MODE == PKV_F32 ? 4 : MODE == PKV_BF16 ? 2 : 1;
  static constexpr int kKeys = MODE == PKV_F32 ? 32 : 64;
  static constexpr int kRow = D * kEs;
  static constexpr int kChunks = kRow / 16;
  static constexpr int kHalf = kKeys * kRow;
  static constexpr int kBytes = 2 * kHalf + (MODE == PKV_I8 ? 2 * kKeys * 16 : 0);
  static constexpr int kStages = kBytes > 16384 ? 3 : 4;
  // Byte offset of chunk c of row r, permuted so that each 8-lane phase of the reads
  // falls in 8 different 16-byte columns.
  static __device__ __forceinline__ int at(int r, int c) {
    if constexpr (MODE == PKV_I8) {
      if constexpr (D == 64) return r * kRow + ((c ^ ((r >> 1) & 3)) << 4);
      return r * kRow + ((c ^ (((r & 1) << 2) | ((r >> 1) & 3))) << 4);
    } else if constexpr (MODE == PKV_F32) {
      return r * kRow + ((c ^ (((r & 6)) ^ ((r & 1) << 2))) << 4);
    }
    return r * kRow + ((c ^ (r & 7)) << 4);
  }
};

// MT: 16-row tiles of a warp; RG: groups of warps that share out a unit's rows.
template <int MODE, int D, int MT, int RG>
struct RowsLayout {
  using Tl = RowsTile<MODE, D>;
  static constexpr int kRows = 16 * MT * RG;
  static constexpr int kRing = Tl::kStages * Tl::kBytes;
  // Q: with two row tiles in shared memory (fp32 as two tf32 parts), with one in registers
  static constexpr bool kQShared = MT > 1;
  static constexpr int kQRow = D * (MODE == PKV_F32 ? 4 : 2);
  static constexpr int kQ = kQShared ? kRows * kQRow * (MODE == PKV_F32 ? 2 : 1) : 0;
  static constexpr int kAccRow = D + 4;  // floats between rows of a merged state
  static constexpr int kMerge = kRowsWarps * 16 * MT * (kAccRow + 2) * 4;
  static constexpr int kQAt = kRing > kMerge ? kRing : kMerge;
  static constexpr int kSeenAt = kQAt + kQ;  // what each of a warp's rows sees
  static constexpr int kSmem = kSeenAt + kRowsWarps * 16 * MT * (int)sizeof(RowSees);
  // CTAs that an SM holds at once, of the tree kernel its grid: what shared memory and O's
  // registers allow
  static constexpr int kFit = 227 * 1024 / (kSmem + 2048);
  static constexpr int kMost = D == 64 || (MODE == PKV_I8 && MT == 1) ? 3 : 2;
  static constexpr int kCtas = kFit < kMost ? kFit : kMost;
};

// One unit's work: rows first_row .. of sequence b, kv head g, tiles t0 .. t1 of its list.
struct RowsPiece {
  SeqSpan s;
  KeyList t;
  int b, g, first_row, t0, t1;
  int lo, hi;    // keys that some row of the unit may see: lo .. hi, and the first ones
  float* part;   // where the state goes, or NULL: finished here
};

template <int MODE, int D, int MT, int RG, bool TREE>
__device__ __forceinline__ void rows_piece(const RowsParams& p, const RowsPiece& w, int ctas,
                                           unsigned char* smem) {
  using Tl = RowsTile<MODE, D>;
  using Lay = RowsLayout<MODE, D, MT, RG>;
  constexpr bool kI8 = MODE == PKV_I8, kF32 = MODE == PKV_F32;
  constexpr int WK = kRowsWarps / RG, KT = Tl::kKeys, KW = KT / WK, NT = KW / 8;
  constexpr int NST = Tl::kStages, M = Lay::kRows, NO = D / 8;
  constexpr bool kTwoParts = MT == 1;  // of a weight in P V
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wr = warp % RG, wk = warp / RG;
  const int gl = lane >> 2, qi = lane & 3;
  const int G = p.plan.G, n = w.s.n, rows = n * G, off = w.s.off;
  const uint32_t base = smem_addr(smem), sq = base + Lay::kQAt;

  // ---- copies: each warp a quarter of a tile's rows ----
  constexpr int RW = KT / kRowsWarps;
  const int sink_end = off + p.plan.span.sink;  // table position
  const int my_r = warp * RW + lane % RW;  // the row of a tile that this lane looks up
  const int32_t* table = p.bt + (long long)w.b * p.plan.span.mb;
  auto seen_by_some = [&](int pos) {
    return pos >= off && pos <= off + w.hi && (pos >= off + w.lo || pos < sink_end);
  };
  auto lookup = [&](int i) -> int {  // block of the lane's row in tile i, INT_MIN: a row of zeros
    if (i >= w.t1) return INT_MIN;
    const int pos = w.t.position(i * KT + my_r);
    return seen_by_some(pos) ? table[pos >> p.bs_bits] : INT_MIN;
  };
  int ahead = lookup(w.t0);
  auto issue = [&](int i, int stage) {
    if (i < w.t1) {
      const int pos = w.t.position(i * KT + my_r);
      int blk = ahead;
      if (blk != INT_MIN && (blk < 0 || blk >= p.num_blocks)) {
        set_error(p.err, kErrIndex);
        blk = INT_MIN;
      }
      const unsigned live = __ballot_sync(kAllLanes, blk != INT_MIN);
      const long long at =
          blk == INT_MIN ? 0
                         : ((((long long)blk * p.L + p.layer) << p.bs_bits) +
                            (pos & ((1 << p.bs_bits) - 1))) * p.row_bytes;
      ahead = lookup(i + 1);
      const uint32_t dst = base + stage * Tl::kBytes;
      constexpr int C = Tl::kChunks;
#pragma unroll
      for (int u = 0; u < RW * C / 32; ++u) {
        const int e = u * 32 + lane, r = e / C, c = e % C;
        const long long src = __shfl_sync(kAllLanes, at, r) + w.g * Tl::kRow + c * 16;
        const bool on = live >> r & 1;
        const uint32_t d = dst + Tl::at(warp * RW + r, c);
        cp_async16(d, p.k + (on ? src : 0), on);
        cp_async16(d + Tl::kHalf, p.v + (on ? src : 0), on);
      }
      if constexpr (kI8) {
        // the 16 bytes that hold the head's scale: lanes 0-15 of K, the others of V
        const bool on = live >> lane & 1;
        const long long src = on ? at + p.scale_off + (4 * w.g & ~15) : 0;
        cp_async16(dst + 2 * Tl::kHalf + (lane / RW * KT + my_r) * 16,
                   (lane < RW ? p.k : p.v) + src, on);
      }
    }
    cp_commit();
  };
#pragma unroll 1
  for (int s = 0; s < NST - 1; ++s) issue(w.t0 + s, s);

  // ---- what the warp's rows see, a row a lane: kept in shared memory ----
  const int warp_row = w.first_row + wr * 16 * MT;
  RowSees* seen_rows = reinterpret_cast<RowSees*>(smem + Lay::kSeenAt) + warp * (16 * MT);
  int full_lo, full_hi;  // places that every row of the warp sees
  {
    const int r = warp_row + lane % (16 * MT);
    const bool live = r < rows;
    const int tok = live ? r / G : 0;
    const RowSees row = row_sees(p.plan.span, w.t, off, w.s.ctx, n, tok, w.s.q0 + tok,
                                 TREE ? p.q_pos : nullptr, TREE ? p.mask : nullptr, p.words);
    if (lane < 16 * MT) seen_rows[lane] = row;
    full_lo = max(row.first, __reduce_max_sync(kAllLanes, live ? row.lo : INT_MIN));
    full_hi = __reduce_min_sync(kAllLanes, live ? row.top : INT_MAX);
    __syncwarp();
  }

  // ---- Q, rows behind the last one as zeros ----
  auto q_row = [&](int r) {
    const int tok = r / G;
    return p.q + ((w.s.q0 + tok) * p.hq + w.g * G + (r - tok * G)) * (long long)Lay::kQRow;
  };
  constexpr int KS = kF32 ? D / 8 : D / 16;
  [[maybe_unused]] uint32_t qa[Lay::kQShared ? 1 : KS][4];
  if constexpr (!Lay::kQShared) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = warp_row + gl + 8 * i;
      const bool live = r < rows;
      const char* src = q_row(live ? r : 0);
      if constexpr (MODE == PKV_BF16) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const char* x = src + (k * 16 + 2 * qi) * 2;
          qa[k][i] = live ? *reinterpret_cast<const uint32_t*>(x) : 0u;
          qa[k][2 + i] = live ? *reinterpret_cast<const uint32_t*>(x + 16) : 0u;
        }
      } else if constexpr (kI8) {
        // step 4 i + j: dims 64 i + 16 qi + 4 j .. + 3, the order of the K codes
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const char* x = src + ((k >> 2) * 64 + 16 * qi + 4 * (k & 3)) * 2;
          const uint2 y = live ? *reinterpret_cast<const uint2*>(x) : make_uint2(0u, 0u);
          qa[k][i] = y.x;
          qa[k][2 + i] = y.y;
        }
      } else {
        // steps 2 i, 2 i + 1: dims 16 i + 4 qi .. + 3
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          const char* x = src + (k * 8 + 4 * qi) * 4;
          const uint4 y = live ? *reinterpret_cast<const uint4*>(x) : make_uint4(0u, 0u, 0u, 0u);
          qa[k][i] = y.x;
          qa[k][2 + i] = y.y;
          qa[k + 1][i] = y.z;
          qa[k + 1][2 + i] = y.w;
        }
      }
    }
  } else {
    // 16-byte chunks; int8: a chunk's two groups of 4 dims (64 i + 16 c + 4 j ..) go where step
    // 4 i + j takes them, columns 2 c, 2 c + 1 and 8 + 2 c, 9 + 2 c of it
    constexpr int C = Lay::kQRow / 16;
#pragma unroll 4
    for (int e = tid; e < M * C; e += kRowsThreads) {
      const int r = e / C, c = e % C;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (w.first_row + r < rows) x = ld_stream(q_row(w.first_row + r) + c * 16);
      const uint32_t at = sq + r * Lay::kQRow;
      if constexpr (MODE == PKV_BF16) {
        sts128(at + ((c ^ (r & 7)) << 4), x);
      } else if constexpr (kI8) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int d = 8 * c + 4 * u, step = (d >> 6) * 4 + ((d >> 2) & 3), col = (d >> 4) & 3;
          sts32(at + (((2 * step) ^ (r & 7)) << 4) + col * 4, u ? x.z : x.x);
          sts32(at + (((2 * step + 1) ^ (r & 7)) << 4) + col * 4, u ? x.w : x.y);
        }
      } else {
        uint4 h, l;
        split_tf32(__uint_as_float(x.x), h.x, l.x);
        split_tf32(__uint_as_float(x.y), h.y, l.y);
        split_tf32(__uint_as_float(x.z), h.z, l.z);
        split_tf32(__uint_as_float(x.w), h.w, l.w);
        sts128(sq + Tl::at(r, c), h);
        sts128(sq + M * Lay::kQRow + Tl::at(r, c), l);
      }
    }
  }
  // the A operand of step k of row tile mt (bf16, int8)
  auto q_frag = [&](int mt, int k, uint32_t (&a)[4]) {
    if constexpr (Lay::kQShared) {
      const int r = wr * 16 * MT + mt * 16 + (lane & 15);
      ldsm_x4(a, sq + r * Lay::kQRow + (((2 * k + (lane >> 4)) ^ (r & 7)) << 4));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) a[c] = qa[k][c];
    }
  };
  // fp32: both parts of steps k, k + 1
  auto q_frag_tf32 = [&](int mt, int k, uint32_t (&h)[2][4], uint32_t (&l)[2][4]) {
    if constexpr (Lay::kQShared) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = wr * 16 * MT + mt * 16 + gl + 8 * i;
        const uint4 x = lds128(sq + Tl::at(r, 2 * k + qi));
        const uint4 y = lds128(sq + M * Lay::kQRow + Tl::at(r, 2 * k + qi));
        h[0][i] = x.x; h[0][2 + i] = x.y; h[1][i] = x.z; h[1][2 + i] = x.w;
        l[0][i] = y.x; l[0][2 + i] = y.y; l[1][i] = y.z; l[1][2 + i] = y.w;
      }
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c) split_tf32(__uint_as_float(qa[k + u][c]), h[u][c], l[u][c]);
    }
  };

  float o[MT][NO][4], m[MT][2], l[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int k = 0; k < NO; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[mt][k][c] = 0.f;
    m[mt][0] = m[mt][1] = -INFINITY;
    l[mt][0] = l[mt][1] = 0.f;
  }

  int stage = 0;
#pragma unroll 1
  for (int i = w.t0; i < w.t1; ++i) {
    cp_wait<NST - 2>();
    __syncthreads();
    issue(i + NST - 1, stage == 0 ? NST - 1 : stage - 1);
    const uint32_t st = base + stage * Tl::kBytes, sv = st + Tl::kHalf;
    if (++stage == NST) stage = 0;
    const int k0 = wk * KW;  // the warp's keys of the tile

    // ---- scores ----
    float s[MT][NT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[mt][j][c] = 0.f;
    if constexpr (MODE == PKV_BF16) {
      const int r = k0 + (lane & 7) + ((lane >> 4) & 1) * 8, cc = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) q_frag(mt, k, a[mt]);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          uint32_t b[4];
          ldsm_x4(b, st + Tl::at(r + j * 8, 2 * k + cc));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16<false>(s[mt][j], a[mt][0], a[mt][1], a[mt][2], a[mt][3], b[0], b[1]);
            mma16<false>(s[mt][j + 1], a[mt][0], a[mt][1], a[mt][2], a[mt][3], b[2], b[3]);
          }
        }
      }
    } else if constexpr (kI8) {
      const int r = k0 + 4 * (gl >> 1) + (gl & 1);
#pragma unroll
      for (int u = 0; u < KS / 4; ++u) {
        uint4 x[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
          x[j] = lds128(st + Tl::at(r + (j >> 1) * 16 + (j & 1) * 2, 4 * u + qi));
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t a[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) q_frag(mt, 4 * u + v, a[mt]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            uint32_t b0, b1;
            codes_to_bf16(v == 0 ? x[j].x : v == 1 ? x[j].y : v == 2 ? x[j].z : x[j].w, b0, b1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              mma16<false>(s[mt][j], a[mt][0], a[mt][1], a[mt][2], a[mt][3], b0, b1);
          }
        }
      }
    } else {
      float big[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) big[mt][j][c] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; k += 2) {
        uint32_t bh[NT][4], bl[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 x = lds128(st + Tl::at(k0 + j * 8 + gl, 2 * k + qi));
          split_tf32(__uint_as_float(x.x), bh[j][0], bl[j][0]);
          split_tf32(__uint_as_float(x.y), bh[j][1], bl[j][1]);
          split_tf32(__uint_as_float(x.z), bh[j][2], bl[j][2]);
          split_tf32(__uint_as_float(x.w), bh[j][3], bl[j][3]);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t ah[2][4], al[2][4];
          q_frag_tf32(mt, k, ah, al);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma8_tf32(s[mt][j], al[u], bh[j][2 * u], bh[j][2 * u + 1]);
              mma8_tf32(s[mt][j], ah[u], bl[j][2 * u], bl[j][2 * u + 1]);
              mma8_tf32(big[mt][j], ah[u], bh[j][2 * u], bh[j][2 * u + 1]);
            }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[mt][j][c] += big[mt][j][c];
    }

    // ---- softmax ----
    // key of column c (0, 1) of score tile j, within the warp's keys
    auto key = [&](int j, int c) {
      if constexpr (kI8) return (j >> 1) * 16 + 4 * qi + (j & 1) * 2 + c;
      return j * 8 + 2 * qi + c;
    };
    const int p0 = i * KT + k0;
    const bool full = p0 >= full_lo && p0 + KW - 1 <= full_hi;
    [[maybe_unused]] float factor[NT][2], scale_v[NT][2];
    if constexpr (kI8) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t sc = st + 2 * Tl::kHalf + (k0 + key(j, c)) * 16 + (4 * w.g & 15);
          factor[j][c] = p.qscale * lds_f32(sc);
          scale_v[j][c] = lds_f32(sc + KT * 16);
        }
    }
    float a[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) s[mt][j][2 * r + c] *= kI8 ? factor[j][c] : p.qscale;
        if (!full) {
          const uint32_t bits = seen_rows[mt * 16 + gl + 8 * r].bits_from(p0) >> key(0, 0);
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (!(bits >> (key(j, c) - key(0, 0)) & 1)) s[mt][j][2 * r + c] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) mx = fmaxf(mx, s[mt][j][2 * r + c]);
        a[mt][r] = 1.f;
        // the running maximum moves only where some lane passes it
        if (__any_sync(kAllLanes, mx > m[mt][r])) {
          mx = fmaxf(mx, __shfl_xor_sync(kAllLanes, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(kAllLanes, mx, 2));
          const float top_m = fmaxf(m[mt][r], mx);
          a[mt][r] = m[mt][r] == -INFINITY ? 0.f : exp2f(m[mt][r] - top_m);
          m[mt][r] = top_m;
        }
        // scores of -inf carry no weight, even while they are all there is
        const float base_m = m[mt][r] == -INFINITY ? 0.f : m[mt][r];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float e = exp2f(s[mt][j][2 * r + c] - base_m);
            sum += e;
            s[mt][j][2 * r + c] = e;
            if constexpr (kI8) s[mt][j][2 * r + c] = e * scale_v[j][c];
          }
        l[mt][r] = l[mt][r] * a[mt][r] + sum;
      }
    if constexpr (!kF32) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        if (__any_sync(kAllLanes, a[mt][0] != 1.f || a[mt][1] != 1.f)) {
#pragma unroll
          for (int k = 0; k < NO; ++k) {
            o[mt][k][0] *= a[mt][0];
            o[mt][k][1] *= a[mt][0];
            o[mt][k][2] *= a[mt][1];
            o[mt][k][3] *= a[mt][1];
          }
        }
    }

    // ---- O += P V ----
    if constexpr (!kF32) {
      uint32_t ph[MT][NT / 2][4];
      [[maybe_unused]] uint32_t pl[MT][NT / 2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < NT / 2; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float x = s[mt][2 * j + (c >> 1)][2 * (c & 1)];
            const float y = s[mt][2 * j + (c >> 1)][2 * (c & 1) + 1];
            if constexpr (!kTwoParts) {
              ph[mt][j][c] = pack_bf16x2(x, y);
            } else {
              if constexpr (kI8) {  // (infinite products: what the finite part leaves is infinite)
                constexpr float kMost = 3.38953139e38f;
                ph[mt][j][c] =
                    pack_bf16x2(fminf(fmaxf(x, -kMost), kMost), fminf(fmaxf(y, -kMost), kMost));
              } else {
                ph[mt][j][c] = below_bf16x2(x, y);
              }
              pl[mt][j][c] = pack_bf16x2(x - bf16_lo(ph[mt][j][c]), y - bf16_hi(ph[mt][j][c]));
            }
          }
      // two output tiles' worth of one V operand
      auto add = [&](int j, int k, uint32_t b0, uint32_t b1) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma16<false>(o[mt][k], ph[mt][j][0], ph[mt][j][1], ph[mt][j][2], ph[mt][j][3], b0, b1);
          if constexpr (kTwoParts)
            mma16<false>(o[mt][k], pl[mt][j][0], pl[mt][j][1], pl[mt][j][2], pl[mt][j][3], b0, b1);
        }
      };
      if constexpr (kI8) {
#pragma unroll
        for (int k = 0; k < NO; k += 2)
#pragma unroll
          for (int j = 0; j < NT / 2; ++j) {
            uint32_t r0, r1, b0, b1, b2, b3;
            ldsm_b8_t(r0, r1, sv + Tl::at(k0 + j * 16 + (lane & 15), k / 2));
            codes_to_bf16(r0, b0, b1);
            codes_to_bf16(r1, b2, b3);
            add(j, k, b0, b1);
            add(j, k + 1, b2, b3);
          }
      } else {
        const int r = k0 + (lane & 7) + ((lane >> 3) & 1) * 8, cc = lane >> 4;
#pragma unroll
        for (int j = 0; j < NT / 2; ++j)
#pragma unroll
          for (int k = 0; k < NO; k += 2) {
            uint32_t b[4];
            ldsm_x4_t(b, sv + Tl::at(r + j * 16, k + cc));
            add(j, k, b[0], b[1]);
            add(j, k + 1, b[2], b[3]);
          }
      }
    } else {
      uint32_t ph[MT][NT][4], pl[MT][NT][4];  // columns qi, qi + 4 of a step: keys 2 qi, 2 qi + 1
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          split_tf32(s[mt][j][0], ph[mt][j][0], pl[mt][j][0]);
          split_tf32(s[mt][j][2], ph[mt][j][1], pl[mt][j][1]);
          split_tf32(s[mt][j][1], ph[mt][j][2], pl[mt][j][2]);
          split_tf32(s[mt][j][3], ph[mt][j][3], pl[mt][j][3]);
        }
      // dims 32 q + 4 column + u of the four output tiles 4 q + u
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint4 x[NT], y[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          x[j] = lds128(sv + Tl::at(k0 + j * 8 + 2 * qi, 8 * q + gl));
          y[j] = lds128(sv + Tl::at(k0 + j * 8 + 2 * qi + 1, 8 * q + gl));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float acc[MT][4], big[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[mt][c] = big[mt][c] = 0.f;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            uint32_t h0, l0, h1, l1;
            split_tf32(__uint_as_float(u == 0 ? x[j].x : u == 1 ? x[j].y : u == 2 ? x[j].z : x[j].w),
                       h0, l0);
            split_tf32(__uint_as_float(u == 0 ? y[j].x : u == 1 ? y[j].y : u == 2 ? y[j].z : y[j].w),
                       h1, l1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma8_tf32(acc[mt], pl[mt][j], h0, h1);
              mma8_tf32(acc[mt], ph[mt][j], l0, l1);
              mma8_tf32(big[mt], ph[mt][j], h0, h1);
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              o[mt][4 * q + u][c] =
                  fmaf(o[mt][4 * q + u][c], a[mt][c >> 1], acc[mt][c] + big[mt][c]);
        }
      }
    }
  }
  cp_wait<0>();
  __syncthreads();

  // four dims of a row's result
  auto finish = [&](int r, int d, float sum, const float (&x)[4]) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no weight at all: zeros
    const int tok = r / G;
    const long long at = ((w.s.q0 + tok) * p.hq + w.g * G + (r - tok * G)) * D + d;
    if constexpr (kF32) {
      *reinterpret_cast<float4*>(p.out + at * 4) =
          make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    } else {
      *reinterpret_cast<uint2*>(p.out + at * 2) =
          make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
    }
    if ((nonfinite(x[0]) || nonfinite(x[1]) || nonfinite(x[2]) || nonfinite(x[3])) && !nonfinite(sum))
      repair_query<4>(p.repair, w.b, tok, w.g * G + (r - tok * G), d, 4);
  };

  // ---- the states to shared memory, and their merge ----
  float* acc = reinterpret_cast<float*>(smem);
  float* ml = acc + kRowsWarps * 16 * MT * Lay::kAccRow;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float sum = l[mt][r];
      sum += __shfl_xor_sync(kAllLanes, sum, 1);
      sum += __shfl_xor_sync(kAllLanes, sum, 2);
      const int row = wk * M + wr * 16 * MT + mt * 16 + gl + 8 * r;
      if (qi == 0) {
        ml[2 * row] = m[mt][r];
        ml[2 * row + 1] = sum;
      }
#pragma unroll
      for (int k = 0; k < NO; ++k) {
        if constexpr (kF32) {
          acc[row * Lay::kAccRow + (k >> 2) * 32 + 8 * qi + (k & 3)] = o[mt][k][2 * r];
          acc[row * Lay::kAccRow + (k >> 2) * 32 + 8 * qi + 4 + (k & 3)] = o[mt][k][2 * r + 1];
        } else {
          *reinterpret_cast<float2*>(acc + row * Lay::kAccRow + k * 8 + 2 * qi) =
              make_float2(o[mt][k][2 * r], o[mt][k][2 * r + 1]);
        }
      }
    }
  __syncthreads();
  if constexpr (!TREE) {
    // prefill: a cluster's CTAs share the unit's tiles, and its rows in their merge
    if (ctas > 1) {
      cluster_sync();
      const uint32_t rank = cluster_rank();
      for (int e = (int)rank * kRowsThreads + tid; e < M * (D / 4); e += ctas * kRowsThreads) {
        const int row = e / (D / 4), d = e % (D / 4) * 4, r = w.first_row + row;
        if (r >= rows) break;
        float top_m = -INFINITY, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < ctas; ++c) {
          const uint32_t ml_c = cluster_map(smem_addr(ml), c), acc_c = cluster_map(base, c);
          float2 s[WK];
          float4 y[WK];
#pragma unroll
          for (int u = 0; u < WK; ++u) {
            s[u] = ld_cluster_f32x2(ml_c + (u * M + row) * 8);
            y[u] = ld_cluster_f32x4(acc_c + ((u * M + row) * Lay::kAccRow + d) * 4);
          }
          float most = top_m;
#pragma unroll
          for (int u = 0; u < WK; ++u) most = fmaxf(most, s[u].x);
          const float shrink = most == top_m ? 1.f : exp2f(top_m - most);
          top_m = most;
          sum *= shrink;
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] *= shrink;
#pragma unroll
          for (int u = 0; u < WK; ++u) {
            // a state at -inf saw nothing, or only NaN: its sum and O are 0, or NaN
            const float f = s[u].x == -INFINITY ? 1.f : exp2f(s[u].x - top_m);
            sum += f * s[u].y;
            x[0] += f * y[u].x;
            x[1] += f * y[u].y;
            x[2] += f * y[u].z;
            x[3] += f * y[u].w;
          }
        }
        finish(r, d, sum, x);
      }
      cluster_sync();  // no CTA leaves while another may still read its states
      return;
    }
  }
  // four dims a thread
  for (int e = tid; e < M * (D / 4); e += kRowsThreads) {
    const int row = e / (D / 4), d = e % (D / 4) * 4, r = w.first_row + row;
    if (r >= rows) break;
    float top_m = -INFINITY;
#pragma unroll
    for (int u = 0; u < WK; ++u) top_m = fmaxf(top_m, ml[2 * (u * M + row)]);
    float sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < WK; ++u) {
      const float mu = ml[2 * (u * M + row)];
      // a state at -inf saw nothing, or only NaN: its sum and O are 0, or NaN
      const float f = mu == -INFINITY ? 1.f : exp2f(mu - top_m);
      sum += f * ml[2 * (u * M + row) + 1];
      const float4 y = *reinterpret_cast<const float4*>(acc + (u * M + row) * Lay::kAccRow + d);
      x[0] += f * y.x;
      x[1] += f * y.y;
      x[2] += f * y.z;
      x[3] += f * y.w;
    }
    if (w.part) {
      float* dst = w.part + (long long)row * (D + 4);
      *reinterpret_cast<float4*>(dst + 4 + d) = make_float4(x[0], x[1], x[2], x[3]);
      if (d == 0) *reinterpret_cast<float2*>(dst) = make_float2(top_m, sum);
      continue;
    }
    finish(r, d, sum, x);
  }
  __syncthreads();  // before the ring is filled again
}

// Tree: the batch's tiles split evenly over the grid (span.cuh).
template <int MODE, int D, int MT, int RG>
__global__ void __launch_bounds__(kRowsThreads, (RowsLayout<MODE, D, MT, RG>::kCtas))
    rows_tree_kernel(const __grid_constant__ RowsParams p) {
  constexpr int KT = RowsTile<MODE, D>::kKeys, M = RowsLayout<MODE, D, MT, RG>::kRows;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long scratch[32];
  griddep_wait();
  griddep_launch_dependents();
  const PlanShare share = plan_share<KT>(p.plan, blockIdx.x, gridDim.x, scratch);
  long long at = share.at, first = share.first;
  const long long end = share.end;
  int b = share.b;
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < p.plan.span.batch; i += blockDim.x)
      if (seq_span(p.plan.span, i).bad) set_error(p.err, kErrCapacity);
  }
  while (at < end) {
    const SeqPlan q = seq_plan<KT>(p.plan, b);
    if (at >= first + q.all_steps) {  // the next sequence
      first += q.all_steps;
      ++b;
      continue;
    }
    const PlanPart part = plan_part(p.plan, q, at - first, end - at);
    at += part.steps;
    if (part.t0 == part.t1) continue;
    RowsPiece w;
    w.s = q.s;
    w.t = q.t;
    w.b = b;
    w.g = part.unit / q.nru;
    w.first_row = (part.unit - w.g * q.nru) * M;
    w.t0 = part.t0;
    w.t1 = part.t1;
    w.lo = window_start(q.s.ctx, p.plan.span.window);
    w.hi = q.s.ctx + q.s.n - 1;
    w.part = nullptr;
    if (w.t0 > 0 || w.t1 < q.t.nt)
      w.part = p.part + (2ll * blockIdx.x + (w.t0 == 0 ? 1 : 0)) * (M * (D + 4));
    rows_piece<MODE, D, MT, RG, true>(p, w, 1, smem);
  }
}

// Prefill: a unit a cluster of CTAs, which take its tiles in turns of equal length; the last
// rows' units first.
template <int MODE, int D, int MT, int RG>
__global__ void __launch_bounds__(kRowsThreads, (RowsLayout<MODE, D, MT, RG>::kCtas))
    rows_prefill_kernel(const __grid_constant__ RowsParams p) {
  constexpr int KT = RowsTile<MODE, D>::kKeys, M = RowsLayout<MODE, D, MT, RG>::kRows;
  extern __shared__ __align__(128) unsigned char smem[];
  griddep_wait();
  griddep_launch_dependents();
  uint32_t ctas;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const int rank = (int)cluster_rank(), item = (int)(blockIdx.x / ctas);
  const int per = p.plan.span.batch * p.plan.hkv;
  const int u = p.units_max - 1 - item / per, rest = item % per;
  RowsPiece w;
  w.b = rest / p.plan.hkv;
  w.g = rest - w.b * p.plan.hkv;
  w.s = seq_span(p.plan.span, w.b);
  if (w.s.bad && u == 0 && w.g == 0 && rank == 0 && threadIdx.x == 0) set_error(p.err, kErrCapacity);
  w.first_row = u * M;
  if (w.first_row >= w.s.n * p.plan.G) return;  // the whole cluster
  const int tok0 = w.first_row / p.plan.G;
  const int tok1 = min(w.s.n - 1, (w.first_row + M - 1) / p.plan.G);
  w.lo = window_start(w.s.ctx + tok0, p.plan.span.window);
  w.hi = w.s.ctx + tok1;
  w.t = key_list<KT>(p.plan.span, w.s.off, w.lo, w.hi);
  w.t0 = (int)((long long)w.t.nt * rank / ctas);
  w.t1 = (int)((long long)w.t.nt * (rank + 1) / ctas);
  w.part = nullptr;
  rows_piece<MODE, D, MT, RG, false>(p, w, (int)ctas, smem);
}

template <int MODE, int D, int MT, int RG>
cudaError_t launch_tree_as(const RowsParams& p, long long grid, int dev, cudaStream_t s) {
  static std::atomic<int> allowed[kDevices];
  const auto kern = rows_tree_kernel<MODE, D, MT, RG>;
  constexpr size_t smem = RowsLayout<MODE, D, MT, RG>::kSmem;
  const cudaError_t e = allow_shared(kern, smem, allowed[dev]);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3((unsigned)grid), dim3(kRowsThreads), smem, s, true, p);
}

// Clusters of as many CTAs as the device holds at once beside one another, with two tiles each
// or more.
template <int MODE, int D, int MT, int RG>
cudaError_t launch_prefill_as(const RowsParams& p, int dev, cudaStream_t s) {
  static std::atomic<int> allowed[kDevices], known[kDevices][kRowsMaxCluster + 1];
  using Lay = RowsLayout<MODE, D, MT, RG>;
  const auto kern = rows_prefill_kernel<MODE, D, MT, RG>;
  cudaError_t e = allow_shared(kern, Lay::kSmem, allowed[dev]);
  if (e != cudaSuccess) return e;
  const long long units = (long long)p.units_max * p.plan.span.batch * p.plan.hkv;
  const long long tiles = (p.keys_most + RowsTile<MODE, D>::kKeys - 1) / RowsTile<MODE, D>::kKeys + 1;
  int ctas = 1;
  for (int c = kRowsMaxCluster; c > 1; c >>= 1) {
    int held = 0;
    e = clusters_held(kern, kRowsThreads, Lay::kSmem, (unsigned)c, known[dev][c], &held);
    if (e != cudaSuccess) return e;
    if (units <= held && tiles >= 2 * c) {
      ctas = c;
      break;
    }
  }
  if (ctas == 1)
    return launch_kernel(kern, dim3((unsigned)units), dim3(kRowsThreads), (size_t)Lay::kSmem, s, true,
                         p);
  return launch_clusters(kern, dim3((unsigned)(units * ctas)), dim3(kRowsThreads), Lay::kSmem,
                         (unsigned)ctas, s, p);
}

// Units of 16, 32 or 64 rows.  A warp holds two row tiles where its registers allow: what it
// reads and converts of K and V then serves both.
template <int MODE, int D>
struct RowsShapes {
  static constexpr int kMT = MODE == PKV_F32 && D == 128 ? 1 : 2;
  using R16 = RowsLayout<MODE, D, 1, 1>;
  using R32 = RowsLayout<MODE, D, kMT, 2 / kMT>;
  using R64 = RowsLayout<MODE, D, kMT, 4 / kMT>;
};

template <int MODE, int D>
cudaError_t launch_rows_d(const RowsParams& p, bool tree, long long grid, int dev, cudaStream_t s) {
  constexpr int MT = RowsShapes<MODE, D>::kMT;
  const int rows = p.plan.unit_rows;
  if (tree)
    return rows == 16   ? launch_tree_as<MODE, D, 1, 1>(p, grid, dev, s)
           : rows == 32 ? launch_tree_as<MODE, D, MT, 2 / MT>(p, grid, dev, s)
                        : launch_tree_as<MODE, D, MT, 4 / MT>(p, grid, dev, s);
  return rows == 16   ? launch_prefill_as<MODE, D, 1, 1>(p, dev, s)
         : rows == 32 ? launch_prefill_as<MODE, D, MT, 2 / MT>(p, dev, s)
                      : launch_prefill_as<MODE, D, MT, 4 / MT>(p, dev, s);
}

template <int MODE, int D>
constexpr int rows_ctas_d(int unit_rows) {
  using S = RowsShapes<MODE, D>;
  return unit_rows == 16 ? S::R16::kCtas : unit_rows == 32 ? S::R32::kCtas : S::R64::kCtas;
}

}  // namespace

// One translation unit a pool type.
cudaError_t launch_rows_bf16(const RowsParams& p, int D, bool tree, long long grid, int dev,
                             cudaStream_t s);
int rows_ctas_bf16(int D, int unit_rows);  // CTAs of the tree kernel that an SM holds
cudaError_t launch_rows_i8(const RowsParams& p, int D, bool tree, long long grid, int dev,
                           cudaStream_t s);
int rows_ctas_i8(int D, int unit_rows);  // CTAs of the tree kernel that an SM holds
cudaError_t launch_rows_f32(const RowsParams& p, int D, bool tree, long long grid, int dev,
                            cudaStream_t s);
int rows_ctas_f32(int D, int unit_rows);  // CTAs of the tree kernel that an SM holds

}  // namespace pkv
