// Attention of several query rows a kv head over one stream of its keys, on mma.sync:
// the general form of pkv_decode_attention_tree and pkv_prefill_attention_window, for
// every pool type, head_dim 64 and 128, any group of heads and block size (prefill.cu
// holds the tcgen05 form for bf16 pools; tree.cu says which call takes which).
//
// What is computed.  The rows of a unit are (new token, query head of kv head g) pairs
// of one sequence, M = 16, 32 or 64 of them.  Softmax attention over the keys that each
// row sees (span.cuh: a window, first tokens, a mask among the new tokens), K and V read
// in place through the block table.
//
// How.  A CTA of 8 warps streams the unit's tiles of KT keys through a ring of 2 or 3
// cp.async stages; rows that no query of the unit sees arrive as zeros, and are not read.
// A tile's scores are shared out by keys (8 or 16 a warp) and, where a tile has fewer
// keys than that, by rows; P then passes through shared memory, and O += P V is shared
// out by dims, an eighth a warp: so no two warps convert or load the same V, and O takes
// M / 16 x D / 64 x 4 registers.  (With keys shared out in both products, four warps a CTA
// and O whole in each, registers held 2 warps a scheduler: 30 tokens on 4096 under a
// window of 4096 35 us instead of 26, an int8 batch of 32 trees 143 instead of 122, fp32
// trees of 32 tokens, D 128, 498 instead of 398; only int8 prompts of D 64 gained by it,
// 186 instead of 235, where a tile has few products for its three barriers.  Two barriers
// a tile, with three stages: 2% less on 64 rows, 3% more on 16.)
//   P is taken against a maximum of the row that moves only when a score passes it by
// more than 8 in log2 units: then, and in the first tile, the warps agree on a new one in
// shared memory; else one __syncthreads_or is all that they exchange.  The sums of a row
// stay in its lanes until the end.
//   bf16: S = Q K^T and O += P V on mma m16n8k16.  Up to 16 rows a weight enters P V as
//     two bf16 parts, within 2^-16 of it together; with more rows, where products are
//     what the kernel spends its time on, as the nearest bf16, as in prefill.cu: off by
//     2^-8 at most, at random, which sums of many keys average out (0.0024 of the
//     result's norm at most was seen against 64 bits, where the output's own rounding is
//     0.0017).
//   int8: fp16 products over the exact codes (to bf16 a code takes three times the
//     instructions of the busiest pipe).  Q is scaled into fp16 by a power of two a row,
//     K's scales are factors of the scores and V's of the weights.  O is kept in units a
//     row in which the largest weight x V scale, at the time that they are chosen, is
//     2^2; they are chosen again with the maximum, and when a V scale passes 2^7 of them
//     (so no product passes 2^15).  A product enters as one fp16, within 2^-11 of it or
//     2^-27 of the largest; up to 16 rows as two, within 2^-22.  (With 2^6 for 2^2 other
//     scales passed 2^7 in most tiles: an int8 prompt took 355 us instead of 301.)  The
//     tile's keys are taken in the order that makes the byte-transposing V load agree
//     with P.
//   fp32: mma m16n8k8 on tf32 in three products: x = hi + lo, each the nearest tf32, and
//     x y ~ hi hi + hi lo + lo hi, within 2^-21 of it.  The tensor cores add with
//     truncation, so the small products have a sum of their own, and O is not their
//     accumulator: each tile's P V is summed from zero and added to O with rounding.
//
// What bounds it.  Few rows of bf16: the keys' bytes (16 trees of 4 tokens on 8192, groups of 4,
// D 128: 89 us, 79 by the bytes; of 8 tokens, D 64, 68 and 40).  int8 (the same trees of 4 tokens
// 88 us, 41 by the bytes), and with more rows, as in fp32, what lies around the products:
// conversions, operands through shared memory, barriers - 50 to 55% of the issue slots and a
// quarter to a third of the tensor pipe.
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
  const unsigned long long* mask;  // tree: [total_q, words], or NULL (tokens see those before)
  int words;
  int* err;
  float* part;  // states of split units
  long long num_blocks;
  int L, layer, row_bytes, scale_off, hq, bs_bits;
  Repair repair;
  int lines;      // tree: 1, or a line of steps a kv head (tree.cu)
  int units_max;  // prefill: units of one kv head of the longest sequence
  long long keys_most;  // prefill: keys that a unit's rows see at most
  float qscale;   // scale * log2(e)
};

constexpr int kRowsWarps = 8;
constexpr int kRowsMaxCluster = 8;
constexpr int kRowsThreads = kRowsWarps * 32;

// Keys of a tile.  int8, 32 rows: 128, so that each K code is converted by one warp only (32
// sequences of 4 to 8 tokens behind 1024 to 8192, 8 kv heads, D 128, G 4: 133 us with 64 keys, 125;
// with 64 rows the scores of 128 keys do not fit in the registers: 325 us where 64 take 301, on
// 4096 tokens of a prompt under a window of 1024).
constexpr int rows_tile_keys(int mode, int rows) {
  return mode == PKV_F32 ? 32 : mode == PKV_I8 && rows == 32 ? 128 : 64;
}

namespace {

constexpr unsigned kAllLanes = 0xffffffffu;
constexpr float kMostUnits = 128.f;  // of a V scale: times a weight of up to 2^8, 2^15 in all

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
template <int MODE, int D, int M>
struct RowsTile {
  static constexpr int kEs = MODE == PKV_F32 ? 4 : MODE == PKV_BF16 ? 2 : 1;
  static constexpr int kKeys = rows_tile_keys(MODE, M);
  static constexpr int kRow = D * kEs;
  static constexpr int kChunks = kRow / 16;
  static constexpr int kHalf = kKeys * kRow;
  static constexpr int kBytes = 2 * kHalf + (MODE == PKV_I8 ? 2 * kKeys * 16 : 0);
  // Byte offset of chunk c of row r, permuted so that each 8-lane phase of the reads
  // falls in 8 different 16-byte columns.
  static __device__ __forceinline__ int at(int r, int c) {
    if constexpr (MODE == PKV_I8) {
      if constexpr (D == 64) return r * kRow + ((c ^ ((r >> 1) & 3)) << 4);
      return r * kRow + ((c ^ (((r & 1) << 2) | ((r >> 1) & 3))) << 4);
    }
    return r * kRow + ((c ^ (r & 7)) << 4);
  }
};

// M: rows of a unit.  The scores of a tile are shared out over the warps by KG groups of 8 keys
// and, where those are fewer than the warps, by row tiles.
template <int MODE, int D, int M>
struct RowsLayout {
  using Tl = RowsTile<MODE, D, M>;
  static constexpr bool kF32 = MODE == PKV_F32;
  static constexpr int KN = M > 16 && !kF32 ? 2 : 1;  // 8-key groups of a warp's scores
  static constexpr int MT = M / 16, KG = Tl::kKeys / 8 / KN, MG = kRowsWarps / KG;
  static constexpr int MS = MT > MG ? MT / MG : 1;  // row tiles of a warp's scores
  static constexpr bool kTwoParts = M == 16 && !kF32;  // of a weight in P V
  // what leaves room for two CTAs an SM
  static constexpr int kStages =
      Tl::kBytes > 32768 || (Tl::kBytes == 32768 && (kF32 || M == 64)) ? 2 : 3;
  static constexpr int kRing = kStages * Tl::kBytes;
  static constexpr int kQRow = D * (kF32 ? 4 : 2), kQPart = M * kQRow;  // fp32: two tf32 parts
  static constexpr int kQAt = kRing;
  static constexpr int kPRow = Tl::kKeys * (kF32 ? 4 : 2), kPPart = M * kPRow;
  static constexpr int kPAt = kQAt + kQPart * (kF32 ? 2 : 1);
  static constexpr int kSeenAt = kPAt + kPPart * (kF32 || kTwoParts ? 2 : 1);
  // of each row: maximum, factor, sum, [KG]; int8 also units, factor of O, [KG]
  static constexpr int kRowAt = kSeenAt + M * (int)sizeof(RowSees);
  static constexpr int kSmem = kRowAt + (3 + KG) * M * 4 + (MODE == PKV_I8 ? (2 + KG) * M * 4 : 0);
  static constexpr int kAccRow = D + 4;  // floats between rows of a state in the merge of a cluster
  static_assert(M * (kAccRow + 2) * 4 <= kRing, "the merge lies over the ring");
  // CTAs that an SM holds at once, of the tree kernel its grid
  static constexpr int kFit = 227 * 1024 / (kSmem + 2048);
  static constexpr int kCtas = kFit < 2 ? kFit : 2;
};

// One unit's work: rows first_row .. of sequence b, kv head g, tiles t0 .. t1 of its list.
struct RowsPiece {
  SeqSpan s;
  KeyList t;
  int b, g, first_row, t0, t1;
  int lo, hi;    // keys that some row of the unit may see: lo .. hi, and the first ones
  float* part;   // where the state goes, or NULL: finished here
};

template <int MODE, int D, int M, bool TREE>
__device__ __forceinline__ void rows_piece(const RowsParams& p, const RowsPiece& w, int ctas,
                                           unsigned char* smem, volatile int* bad_entry = nullptr) {
  using Tl = RowsTile<MODE, D, M>;
  using Lay = RowsLayout<MODE, D, M>;
  constexpr bool kI8 = MODE == PKV_I8, kF32 = MODE == PKV_F32, kTwoParts = Lay::kTwoParts;
  constexpr int KT = Tl::kKeys, NST = Lay::kStages, MT = Lay::MT, MS = Lay::MS, KG = Lay::KG;
  constexpr int KN = Lay::KN, KS = kF32 ? D / 8 : D / 16;         // steps of a score
  constexpr int NO = D / kRowsWarps / 8;            // 8-dim output tiles of a warp
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // scores: KN groups of 8 keys from KN kg, row tiles from mg MS
  const int kg = warp % KG, mg = warp / KG;
  const bool scores = mg * MS < MT;
  const int gl = lane >> 2, qi = lane & 3;
  const int G = p.plan.G, n = w.s.n, rows = n * G, off = w.s.off;
  const uint32_t base = smem_addr(smem), sq = base + Lay::kQAt, sp = base + Lay::kPAt;
  RowSees* seen_rows = reinterpret_cast<RowSees*>(smem + Lay::kSeenAt);
  float* row_max = reinterpret_cast<float*>(smem + Lay::kRowAt);  // [M]: what P is taken against
  float* row_factor = row_max + M;                                // [M]: of O, when it moved
  float* row_sum = row_factor + M;                                // [M]: at the end
  float* row_part = row_sum + M;                                  // [KG][M]
  // int8: O is in units of 2^row_units (in the scores' base), so that weight x V scale fits fp16
  [[maybe_unused]] float* row_units = row_part + KG * M;
  [[maybe_unused]] float* row_factor_o = row_units + M;
  [[maybe_unused]] float* row_top = row_factor_o + M;  // [KG][M]

  // ---- copies: each warp an eighth of a tile's rows ----
  constexpr int RW = KT / kRowsWarps;
  const int sink_end = off + p.plan.span.sink;  // table position
  const int my_r = warp * RW + lane % RW;  // the row of a tile that this lane looks up
  const int32_t* table = p.bt + (long long)w.b * p.plan.span.mb;
  auto seen_by_some = [&](int pos) {
    return pos >= off && pos <= off + w.hi && (pos >= off + w.lo || pos < sink_end);
  };
  // block of the lane's row in tile i; INT_MIN: a row of zeros
  auto lookup = [&](int i) -> int {
    if (i >= w.t1) return INT_MIN;
    const int pos = w.t.position(i * KT + my_r);
    return seen_by_some(pos) ? table[pos >> p.bs_bits] : INT_MIN;
  };
  auto issue = [&](int i, int stage, int blk, auto look) {
    if (i < w.t1) {
      const int pos = w.t.position(i * KT + my_r);
      if (blk < 0 || blk >= p.num_blocks) {
        if (seen_by_some(pos)) {  // (an entry may hold any number, INT_MIN too)
          if constexpr (TREE)
            *bad_entry = 1;  // looked into at the end
          else
            set_error(p.err, kErrIndex);
        }
        blk = INT_MIN;
      }
      const unsigned live = __ballot_sync(kAllLanes, blk != INT_MIN);
      const long long at =
          blk == INT_MIN ? 0
                         : ((((long long)blk * p.L + p.layer) << p.bs_bits) +
                            (pos & ((1 << p.bs_bits) - 1))) * p.row_bytes;
      const uint32_t dst = base + stage * Tl::kBytes;
      look();
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
        // the 16 bytes that hold the head's scale: lanes 0-7 of K, 8-15 of V
        const bool on = live >> lane & 1;
        const long long src = on ? at + p.scale_off + (4 * w.g & ~15) : 0;
        if (lane < 2 * RW)
          cp_async16(dst + 2 * Tl::kHalf + (lane / RW * KT + my_r) * 16,
                     (lane < RW ? p.k : p.v) + src, on);
      }
    }
    cp_commit();
  };
  static_assert(RW * Tl::kChunks >= 32, "every lane copies");
  int ahead[NST];  // looked up together
#pragma unroll
  for (int s = 0; s < NST; ++s) ahead[s] = lookup(w.t0 + s);
#pragma unroll
  for (int s = 0; s < NST - 1; ++s) issue(w.t0 + s, s, ahead[s], [] {});
  int next = ahead[NST - 1];  // of the tile that is copied next

  // ---- what the rows see: kept in shared memory, and the places that all of them see ----
  int full_lo = INT_MIN, full_hi = INT_MAX;
  for (int r0 = 0; r0 < M; r0 += 32) {
    const int r = w.first_row + r0 + lane;
    const bool live = r0 + lane < M && r < rows;
    const int tok = live ? r / G : 0;
    const RowSees row = row_sees(p.plan.span, w.t, off, w.s.ctx, n, tok, w.s.q0 + tok,
                                 TREE ? p.q_pos : nullptr, TREE ? p.mask : nullptr, p.words);
    if (r0 + lane < M && warp == (r0 >> 5)) seen_rows[r0 + lane] = row;
    full_lo = max(full_lo, max(row.first, __reduce_max_sync(kAllLanes, live ? row.lo : INT_MIN)));
    full_hi = min(full_hi, __reduce_min_sync(kAllLanes, live ? row.top : INT_MAX));
  }
  if (tid < M) {
    row_max[tid] = -INFINITY;
    if constexpr (kI8) row_units[tid] = -INFINITY;
  }

  // ---- Q to shared memory, rows behind the last one as zeros ----
  auto q_row = [&](int r) {
    const int tok = r / G;
    return p.q + ((w.s.q0 + tok) * p.hq + w.g * G + (r - tok * G)) * (long long)Lay::kQRow;
  };
  {
    // 16-byte chunks; int8: a chunk's two groups of 4 dims (64 i + 16 c + 4 j ..) go where step
    // 4 i + j takes them, columns 2 c, 2 c + 1 and 8 + 2 c, 9 + 2 c of it: the order of the K codes
    constexpr int C = Lay::kQRow / 16;
    static_assert(C <= 32 && M * C % 32 == 0, "a row's chunks lie in one warp");
    [[maybe_unused]] float* q_unit = row_sum;  // until the end
#pragma unroll 4
    for (int e = tid; e < M * C; e += kRowsThreads) {
      const int r = e / C, c = e % C;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (w.first_row + r < rows) x = ld_stream(q_row(w.first_row + r) + c * 16);
      const uint32_t at = sq + r * Lay::kQRow;
      if constexpr (MODE == PKV_BF16) {
        sts128(at + ((c ^ (r & 7)) << 4), x);
      } else if constexpr (kI8) {
        // fp16, in units of a power of two that puts the row's largest in 2^14 .. 2^15: exact, but
        // for what lies under 2^-39 of the largest (infinities stay)
        int top = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t word = u < 2 ? x.x : u < 4 ? x.y : u < 6 ? x.z : x.w;
          const int e = (word >> (16 * (u & 1) + 7)) & 255;
          if (e != 255) top = max(top, e);
        }
#pragma unroll
        for (int u = 1; u < C; u <<= 1) top = max(top, __shfl_xor_sync(kAllLanes, top, u));
        top = max(top, 40);  // (no unit under 2^-101)
        const float up = __int_as_float((141 - top + 127) << 23);
        if (c == 0) q_unit[r] = __int_as_float((top - 141 + 127) << 23);
        x.x = pack_f16x2(bf16_lo(x.x) * up, bf16_hi(x.x) * up);
        x.y = pack_f16x2(bf16_lo(x.y) * up, bf16_hi(x.y) * up);
        x.z = pack_f16x2(bf16_lo(x.z) * up, bf16_hi(x.z) * up);
        x.w = pack_f16x2(bf16_lo(x.w) * up, bf16_hi(x.w) * up);
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
        sts128(at + ((c ^ (r & 7)) << 4), h);
        sts128(at + Lay::kQPart + ((c ^ (r & 7)) << 4), l);
      }
    }
  }
  // An A operand of 16 rows and two 16-byte chunks (16 columns of 16 bits, 8 of tf32) of Q or P.
  auto a_frag = [&](uint32_t from, int row_bytes, int mt, int step, uint32_t (&a)[4]) {
    const int r = mt * 16 + (lane & 15);
    ldsm_x4(a, from + r * row_bytes + (((2 * step + (lane >> 4)) ^ (r & 7)) << 4));
  };

  float o[MT][NO][4], m[MS][2], l[MS][2];
  [[maybe_unused]] float unit[MS][2], q_unit[MS][2];
  if constexpr (kI8) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < MS; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        unit[j][r] = 1.f;
        q_unit[j][r] = scores ? row_sum[(mg * MS + j) * 16 + gl + 8 * r] * p.qscale : 0.f;
      }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int k = 0; k < NO; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[mt][k][c] = 0.f;
#pragma unroll
  for (int i = 0; i < MS; ++i) {
    m[i][0] = m[i][1] = -INFINITY;
    l[i][0] = l[i][1] = 0.f;
  }

  int stage = 0;
#pragma unroll 1
  for (int i = w.t0; i < w.t1; ++i) {
    cp_wait<NST - 2>();
    __syncthreads();  // the tile is there, and the last one's P and stage are done with
    issue(i + NST - 1, stage == 0 ? NST - 1 : stage - 1, next, [&] { next = lookup(i + NST); });
    const uint32_t st = base + stage * Tl::kBytes, sv = st + Tl::kHalf;
    if (++stage == NST) stage = 0;

    // ---- the warp's scores ----
    float s[MS][KN][4];
    [[maybe_unused]] float scale_v[KN][2];
    bool raise = false;
    if (scores) {
#pragma unroll
      for (int j = 0; j < MS; ++j)
#pragma unroll
        for (int e = 0; e < KN; ++e)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[j][e][c] = 0.f;
      if constexpr (MODE == PKV_BF16) {
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          uint32_t b[KN][4];
#pragma unroll
          for (int e = 0; e < KN; ++e)
            ldsm_x4(b[e], st + Tl::at((kg * KN + e) * 8 + (lane & 7), 2 * k + (lane >> 3)));
#pragma unroll
          for (int j = 0; j < MS; ++j)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t a[4];
              a_frag(sq, Lay::kQRow, mg * MS + j, k + u, a);
#pragma unroll
              for (int e = 0; e < KN; ++e)
                mma16<false>(s[j][e], a[0], a[1], a[2], a[3], b[e][2 * u], b[e][2 * u + 1]);
            }
        }
      } else if constexpr (kI8) {
#pragma unroll
        for (int u = 0; u < KS / 4; ++u) {
          uint4 x[KN];
#pragma unroll
          for (int e = 0; e < KN; ++e)
            x[e] = lds128(st + Tl::at((kg * KN + e) * 8 + gl, 4 * u + qi));
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t b[KN][2];
#pragma unroll
            for (int e = 0; e < KN; ++e)
              codes_to_f16(v == 0 ? x[e].x : v == 1 ? x[e].y : v == 2 ? x[e].z : x[e].w, b[e][0],
                            b[e][1]);
#pragma unroll
            for (int j = 0; j < MS; ++j) {
              uint32_t a[4];
              a_frag(sq, Lay::kQRow, mg * MS + j, 4 * u + v, a);
#pragma unroll
              for (int e = 0; e < KN; ++e)
                mma16<true>(s[j][e], a[0], a[1], a[2], a[3], b[e][0], b[e][1]);
            }
          }
        }
      } else {
        float big[MS][4];
#pragma unroll
        for (int j = 0; j < MS; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) big[j][c] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          uint32_t b[4], bh[4], bl[4];
          ldsm_x4(b, st + Tl::at(kg * 8 + (lane & 7), 2 * k + (lane >> 3)));
#pragma unroll
          for (int c = 0; c < 4; ++c) split_tf32(__uint_as_float(b[c]), bh[c], bl[c]);
#pragma unroll
          for (int j = 0; j < MS; ++j)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t ah[4], al[4];
              a_frag(sq, Lay::kQRow, mg * MS + j, k + u, ah);
              a_frag(sq + Lay::kQPart, Lay::kQRow, mg * MS + j, k + u, al);
              mma8_tf32(s[j][0], al, bh[2 * u], bh[2 * u + 1]);
              mma8_tf32(s[j][0], ah, bl[2 * u], bl[2 * u + 1]);
              mma8_tf32(big[j], ah, bh[2 * u], bh[2 * u + 1]);
            }
        }
#pragma unroll
        for (int j = 0; j < MS; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[j][0][c] += big[j][c];
      }
      // scaled, masked, and looked at: P is taken against a maximum that moves only when a score
      // passes it by more than 8 (in log2 units, so P stays below 2^8)
#pragma unroll
      for (int e = 0; e < KN; ++e) {
        [[maybe_unused]] float f[2];
        if constexpr (kI8) {
          const uint32_t sc =
              st + 2 * Tl::kHalf + ((kg * KN + e) * 8 + 2 * qi) * 16 + (4 * w.g & 15);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            f[c] = lds_f32(sc + c * 16);
            scale_v[e][c] = lds_f32(sc + (KT + c) * 16);
          }
        }
        const int x0 = i * KT + (kg * KN + e) * 8;
        const bool full = x0 >= full_lo && x0 + 7 <= full_hi;
#pragma unroll
        for (int j = 0; j < MS; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float &x = s[j][e][2 * r], &y = s[j][e][2 * r + 1];
            if constexpr (kI8) {
              x *= q_unit[j][r] * f[0];
              y *= q_unit[j][r] * f[1];
            } else {
              x *= p.qscale;
              y *= p.qscale;
            }
            if (!full) {
              const uint32_t bits =
                  seen_rows[(mg * MS + j) * 16 + gl + 8 * r].bits_from(x0) >> (2 * qi);
              if (!(bits & 1)) x = -INFINITY;
              if (!(bits & 2)) y = -INFINITY;
            }
            raise |= fmaxf(x, y) > m[j][r] + 8.f;
            if constexpr (kI8)
              raise |= fmaxf(fabsf(scale_v[e][0]), fabsf(scale_v[e][1])) * unit[j][r] > kMostUnits;
          }
      }
    }
    if (__syncthreads_or(raise)) {
      // the rows' new maxima, agreed on through shared memory
      if (scores) {
#pragma unroll
        for (int j = 0; j < MS; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float x = fmaxf(s[j][0][2 * r], s[j][0][2 * r + 1]);
            if constexpr (KN == 2) x = fmaxf(x, fmaxf(s[j][1][2 * r], s[j][1][2 * r + 1]));
            x = fmaxf(x, __shfl_xor_sync(kAllLanes, x, 1));
            x = fmaxf(x, __shfl_xor_sync(kAllLanes, x, 2));
            if (qi == 0) row_part[kg * M + (mg * MS + j) * 16 + gl + 8 * r] = x;
            if constexpr (kI8) {
              float top = -INFINITY;  // of weight x V scale
#pragma unroll
              for (int e = 0; e < KN; ++e)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const float f = log2f(fabsf(scale_v[e][c]));
                  if (f < 129.f) top = fmaxf(top, s[j][e][2 * r + c] + f);
                }
              top = fmaxf(top, __shfl_xor_sync(kAllLanes, top, 1));
              top = fmaxf(top, __shfl_xor_sync(kAllLanes, top, 2));
              if (qi == 0) row_top[kg * M + (mg * MS + j) * 16 + gl + 8 * r] = top;
            }
          }
      }
      __syncthreads();
      if (tid < M) {
        const float old = row_max[tid];
        float x = old;
#pragma unroll
        for (int u = 0; u < KG; ++u) x = fmaxf(x, row_part[u * M + tid]);
        row_max[tid] = x;
        row_factor[tid] = old == -INFINITY ? 0.f : exp2f(old - x);
        if constexpr (kI8) {
          const float before = row_units[tid];
          float top = fmaxf(before, x - 110.f);
#pragma unroll
          for (int u = 0; u < KG; ++u) top = fmaxf(top, row_top[u * M + tid] - 2.f);
          row_units[tid] = top;
          row_factor_o[tid] = before == -INFINITY ? 0.f : exp2f(before - top);
        }
      }
      __syncthreads();
      if (scores) {
#pragma unroll
        for (int j = 0; j < MS; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = (mg * MS + j) * 16 + gl + 8 * r;
            m[j][r] = row_max[row];
            l[j][r] *= row_factor[row];
            if constexpr (kI8)
              unit[j][r] = m[j][r] == -INFINITY ? 1.f : exp2f(m[j][r] - row_units[row]);
          }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float a = (kI8 ? row_factor_o : row_factor)[mt * 16 + gl + 8 * r];
#pragma unroll
          for (int k = 0; k < NO; ++k) {
            o[mt][k][2 * r] *= a;
            o[mt][k][2 * r + 1] *= a;
          }
        }
    }
    // ---- P to shared memory, in the order in which the products below take the keys ----
    if (scores) {
#pragma unroll
      for (int j = 0; j < MS; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < KN; ++e) {
          const int grp = kg * KN + e;
          const int row = (mg * MS + j) * 16 + gl + 8 * r;
          // scores of -inf carry no weight, even while they are all there is
          const float mr = m[j][r] == -INFINITY ? 0.f : m[j][r];
          float x = exp2f(s[j][e][2 * r] - mr), y = exp2f(s[j][e][2 * r + 1] - mr);
          l[j][r] += x + y;
          const uint32_t at = sp + row * Lay::kPRow;
          if constexpr (kF32) {
            // keys 2 t, 2 t + 1 of the group: columns t, t + 4
            uint32_t h, lo;
            split_tf32(x, h, lo);
            sts32(at + (((2 * grp) ^ (row & 7)) << 4) + qi * 4, h);
            sts32(at + Lay::kPPart + (((2 * grp) ^ (row & 7)) << 4) + qi * 4, lo);
            split_tf32(y, h, lo);
            sts32(at + (((2 * grp + 1) ^ (row & 7)) << 4) + qi * 4, h);
            sts32(at + Lay::kPPart + (((2 * grp + 1) ^ (row & 7)) << 4) + qi * 4, lo);
          } else {
            int chunk = grp, col = qi * 4;
            if constexpr (kI8) {
              // keys 4 T + u of 16: columns 2 T + u, and 8 + 2 T + u - 2 from u = 2 on
              x = x * unit[j][r] * scale_v[e][0];
              y = y * unit[j][r] * scale_v[e][1];
              chunk = 2 * (grp >> 1) + (qi & 1);
              col = (2 * (grp & 1) + (qi >> 1)) * 4;
            }
            uint32_t h;
            if constexpr (!kTwoParts) {
              h = kI8 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
            } else {
              uint32_t rest;
              if constexpr (kI8) {
                h = pack_f16x2_finite(x, y);
                const float2 f = unpack_f16x2(h);
                rest = pack_f16x2(x - f.x, y - f.y);
              } else {
                h = below_bf16x2(x, y);
                rest = pack_bf16x2(x - bf16_lo(h), y - bf16_hi(h));
              }
              sts32(at + Lay::kPPart + ((chunk ^ (row & 7)) << 4) + col, rest);
            }
            sts32(at + ((chunk ^ (row & 7)) << 4) + col, h);
          }
        }
    }
    __syncthreads();

    // ---- O += P V: every warp all keys, D / 8 of the dims ----
    if constexpr (!kF32) {
#pragma unroll
      for (int k = 0; k < KT / 16; ++k) {
        uint32_t b[NO][2];
        if constexpr (kI8) {
          uint32_t r0, r1;
          ldsm_b8_t(r0, r1, sv + Tl::at(k * 16 + (lane & 15), NO == 2 ? warp : warp >> 1));
          if constexpr (NO == 2) {
            codes_to_f16(r0, b[0][0], b[0][1]);
            codes_to_f16(r1, b[1][0], b[1][1]);
          } else {
            codes_to_f16(warp & 1 ? r1 : r0, b[0][0], b[0][1]);
          }
        } else if constexpr (NO == 2) {
          uint32_t v[4];
          ldsm_x4_t(v, sv + Tl::at(k * 16 + (lane & 15), 2 * warp + (lane >> 4)));
          b[0][0] = v[0]; b[0][1] = v[1]; b[1][0] = v[2]; b[1][1] = v[3];
        } else {
          ldsm_x2_t(b[0][0], b[0][1], sv + Tl::at(k * 16 + (lane & 15), warp));
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t a[4];
          a_frag(sp, Lay::kPRow, mt, k, a);
#pragma unroll
          for (int u = 0; u < NO; ++u)
            mma16<kI8>(o[mt][u], a[0], a[1], a[2], a[3], b[u][0], b[u][1]);
          if constexpr (kTwoParts) {
            a_frag(sp + Lay::kPPart, Lay::kPRow, mt, k, a);
#pragma unroll
            for (int u = 0; u < NO; ++u)
              mma16<kI8>(o[mt][u], a[0], a[1], a[2], a[3], b[u][0], b[u][1]);
          }
        }
      }
    } else {
      // dims NO column + u of the warp's output tile u
      float acc[MT][NO][4], big[MT][NO][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int u = 0; u < NO; ++u)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[mt][u][c] = big[mt][u][c] = 0.f;
#pragma unroll
      for (int k = 0; k < KT / 8; ++k) {
        uint32_t h[NO][2], lo[NO][2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = k * 8 + 2 * qi + c, byte = (warp * NO * 8 + gl * NO) * 4;
          const uint32_t at = sv + Tl::at(r, byte >> 4) + (byte & 15);
          if constexpr (NO == 2) {
            const float2 x = lds_f32x2(at);
            split_tf32(x.x, h[0][c], lo[0][c]);
            split_tf32(x.y, h[1][c], lo[1][c]);
          } else {
            split_tf32(lds_f32(at), h[0][c], lo[0][c]);
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t ah[4], al[4];
          a_frag(sp, Lay::kPRow, mt, k, ah);
          a_frag(sp + Lay::kPPart, Lay::kPRow, mt, k, al);
#pragma unroll
          for (int u = 0; u < NO; ++u) {
            mma8_tf32(acc[mt][u], al, h[u][0], h[u][1]);
            mma8_tf32(acc[mt][u], ah, lo[u][0], lo[u][1]);
            mma8_tf32(big[mt][u], ah, h[u][0], h[u][1]);
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int u = 0; u < NO; ++u)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[mt][u][c] += acc[mt][u][c] + big[mt][u][c];
    }
  }
  cp_wait<0>();

  // ---- the rows' sums ----
  if (scores) {
#pragma unroll
    for (int j = 0; j < MS; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = l[j][r];
        x += __shfl_xor_sync(kAllLanes, x, 1);
        x += __shfl_xor_sync(kAllLanes, x, 2);
        if (qi == 0) row_part[kg * M + (mg * MS + j) * 16 + gl + 8 * r] = x;
      }
  }
  __syncthreads();
  if (tid < M) {
    float x = 0.f;
#pragma unroll
    for (int u = 0; u < KG; ++u) x += row_part[u * M + tid];
    row_sum[tid] = x;
    row_factor[tid] = 0.f;  // from here on: 1 where the row is to be computed again
  }
  __syncthreads();
  if constexpr (kI8) {  // O in units of 1
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = mt * 16 + gl + 8 * r;
        const float a = row_max[row] == -INFINITY ? 1.f : exp2f(row_units[row] - row_max[row]);
#pragma unroll
        for (int k = 0; k < NO; ++k) {
          o[mt][k][2 * r] *= a;
          o[mt][k][2 * r + 1] *= a;
        }
      }
  }
  // N dims from d on of row r's result
  bool spoiled = false;
  auto finish = [&](int r, int d, float sum, const auto& x) {
    constexpr int N = sizeof(x) / sizeof(x[0]);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no weight at all: zeros
    const int tok = r / G;
    const long long at = ((w.s.q0 + tok) * p.hq + w.g * G + (r - tok * G)) * D + d;
    bool finite = true;
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      if constexpr (kF32)
        *reinterpret_cast<float2*>(p.out + (at + e) * 4) = make_float2(x[e] * inv, x[e + 1] * inv);
      else
        *reinterpret_cast<uint32_t*>(p.out + (at + e) * 2) =
            pack_bf16x2(x[e] * inv, x[e + 1] * inv);
      finite &= !nonfinite(x[e]) && !nonfinite(x[e + 1]);
    }
    if (!finite && !nonfinite(sum)) {
      spoiled = true;
      row_factor[r - w.first_row] = 1.f;
    }
  };
  // over the whole CTA, and a barrier of it: the rows that a value outside them spoiled (repair.cuh)
  auto repair_spoiled = [&] {
    if (!__syncthreads_or(spoiled)) return;
    for (int row = warp; row < M; row += kRowsWarps) {
      if (row_factor[row] == 0.f) continue;
      const int r = w.first_row + row, tok = r / G;
      repair_row<MODE, 1>(p.repair, w.b, tok, w.g * G + (r - tok * G));
    }
    __syncthreads();
  };
  // this warp's values of a row: dim(u, c) is column c of output tile u
  auto dim = [&](int u, int c) {
    if constexpr (kF32) return warp * NO * 8 + (2 * qi + c) * NO + u;
    return warp * NO * 8 + u * 8 + 2 * qi + c;
  };
  const bool cluster = !TREE && ctas > 1;
  float* acc = reinterpret_cast<float*>(smem);  // a cluster: [M][kAccRow], over the ring
  float2* state = reinterpret_cast<float2*>(acc + M * Lay::kAccRow);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int r8 = 0; r8 < 2; ++r8) {
      const int row = mt * 16 + gl + 8 * r8, r = w.first_row + row;
      if (r >= rows) continue;
      float* dst = cluster  ? acc + row * Lay::kAccRow
                   : w.part ? w.part + (long long)row * (D + 4) + 4
                            : nullptr;
      if (dst) {
#pragma unroll
        for (int u = 0; u < NO; ++u)
#pragma unroll
          for (int c = 0; c < 2; ++c) dst[dim(u, c)] = o[mt][u][2 * r8 + c];
      } else if constexpr (kF32 && NO == 2) {
        const float x[4] = {o[mt][0][2 * r8], o[mt][1][2 * r8], o[mt][0][2 * r8 + 1],
                            o[mt][1][2 * r8 + 1]};
        finish(r, dim(0, 0), row_sum[row], x);
      } else {
#pragma unroll
        for (int u = 0; u < NO; ++u) {
          const float x[2] = {o[mt][u][2 * r8], o[mt][u][2 * r8 + 1]};
          finish(r, dim(u, 0), row_sum[row], x);
        }
      }
    }
  if (w.part && tid < M && w.first_row + tid < rows)
    *reinterpret_cast<float2*>(w.part + (long long)tid * (D + 4)) =
        make_float2(row_max[tid], row_sum[tid]);
  if constexpr (!TREE) {
    // prefill: a cluster's CTAs share the unit's tiles, and its rows in their merge
    if (ctas > 1) {
      if (tid < M) state[tid] = make_float2(row_max[tid], row_sum[tid]);
      cluster_sync();
      const uint32_t rank = cluster_rank();
      for (int e = (int)rank * kRowsThreads + tid; e < M * (D / 4); e += ctas * kRowsThreads) {
        const int row = e / (D / 4), d = e % (D / 4) * 4, r = w.first_row + row;
        if (r >= rows) break;
        float top = -INFINITY, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
        float2 ml[kRowsMaxCluster];
        float4 y[kRowsMaxCluster];
#pragma unroll
        for (int c = 0; c < kRowsMaxCluster; ++c) {
          ml[c] = make_float2(-INFINITY, 0.f);
          y[c] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c < ctas) {
            ml[c] = ld_cluster_f32x2(cluster_map(smem_addr(state + row), c));
            y[c] = ld_cluster_f32x4(cluster_map(smem_addr(acc + row * Lay::kAccRow + d), c));
          }
          top = fmaxf(top, ml[c].x);
        }
#pragma unroll
        for (int c = 0; c < kRowsMaxCluster; ++c) {
          // a state at -inf saw nothing, or only NaN: its sum and O are 0, or NaN
          const float f = ml[c].x == -INFINITY ? 1.f : exp2f(ml[c].x - top);
          sum += f * ml[c].y;
          x[0] += f * y[c].x;
          x[1] += f * y[c].y;
          x[2] += f * y[c].z;
          x[3] += f * y[c].w;
        }
        finish(r, d, sum, x);
      }
      repair_spoiled();
      cluster_sync();  // no CTA leaves while another may still read its states
      return;
    }
  }
  repair_spoiled();  // (a barrier, too, before the ring is filled again)
  if constexpr (TREE) {
    if (*bad_entry) {  // a table entry outside the pool
      for (int x = w.t0 * KT + tid; x < w.t1 * KT; x += kRowsThreads) {
        const int pos = w.t.position(x), e = pos >> p.bs_bits;
        if (!seen_by_some(pos) || (x > w.t0 * KT && w.t.position(x - 1) >> p.bs_bits == e)) continue;
        const int blk = table[e];
        if (blk < 0 || blk >= p.num_blocks)
          report_entry(p.plan.span, p.q_pos, p.mask, p.words, w.b, e, p.err);
      }
      __syncthreads();
      if (tid == 0) *bad_entry = 0;
      __syncthreads();
    }
  }
}

// Tree: the batch's tiles split evenly over the grid (span.cuh).
template <int MODE, int D, int M>
__global__ void __launch_bounds__(kRowsThreads, (RowsLayout<MODE, D, M>::kCtas))
    rows_tree_kernel(const __grid_constant__ RowsParams p) {
  constexpr int KT = RowsTile<MODE, D, M>::kKeys;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long scratch[32];
  __shared__ int bad_entry;
  if (threadIdx.x == 0) bad_entry = 0;
  griddep_wait();
  griddep_launch_dependents();
  const int line_of = (int)blockIdx.x % p.lines;
  const PlanShare share =
      plan_share<KT>(p.plan, (int)blockIdx.x / p.lines, (int)gridDim.x / p.lines, scratch);
  // where the CTA is, kept in shared memory: registers that a piece's work wants for itself
  volatile long long* line = scratch;  // at, first, end, b
  __syncthreads();
  if (threadIdx.x == 0) {
    line[0] = share.at;
    line[1] = share.first;
    line[2] = share.end;
    line[3] = share.b;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < p.plan.span.batch; i += blockDim.x)
      if (seq_span(p.plan.span, i).bad) set_error(p.err, kErrCapacity);
  }
  for (;;) {
    long long at = line[0], first = line[1];
    const long long end = line[2];
    int b = (int)line[3];
    if (at >= end) break;
    SeqPlan q = seq_plan<KT>(p.plan, b);
    while (at >= first + q.all_steps) {  // the next sequence
      first += q.all_steps;
      q = seq_plan<KT>(p.plan, ++b);
    }
    const PlanPart part = plan_part(p.plan, q, at - first, end - at);
    __syncthreads();
    if (threadIdx.x == 0) {
      line[0] = at + part.steps;
      line[1] = first;
      line[3] = b;
    }
    __syncthreads();
    if (part.t0 == part.t1) continue;
    RowsPiece w;
    w.s = q.s;
    w.t = q.t;
    w.b = b;
    const int g = part.unit / q.nru;  // (0 where each kv head has its line)
    w.g = line_of + g;
    w.first_row = (part.unit - g * q.nru) * M;
    w.t0 = part.t0;
    w.t1 = part.t1;
    w.lo = window_start(q.s.ctx, p.plan.span.window);
    w.hi = q.s.ctx + q.s.n - 1;
    w.part = nullptr;
    if (w.t0 > 0 || w.t1 < q.t.nt)
      w.part = p.part + (2ll * blockIdx.x + (w.t0 == 0 ? 1 : 0)) * (M * (D + 4));
    rows_piece<MODE, D, M, true>(p, w, 1, smem, &bad_entry);
  }
}

// Prefill: a unit a cluster of CTAs, which take its tiles in turns of equal length; the last
// rows' units first.
template <int MODE, int D, int M>
__global__ void __launch_bounds__(kRowsThreads, (RowsLayout<MODE, D, M>::kCtas))
    rows_prefill_kernel(const __grid_constant__ RowsParams p) {
  constexpr int KT = RowsTile<MODE, D, M>::kKeys;
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
  rows_piece<MODE, D, M, false>(p, w, (int)ctas, smem);
}

template <int MODE, int D, int M>
cudaError_t launch_tree_as(const RowsParams& p, long long grid, int dev, cudaStream_t s) {
  static std::atomic<int> allowed[kDevices];
  const auto kern = rows_tree_kernel<MODE, D, M>;
  constexpr size_t smem = RowsLayout<MODE, D, M>::kSmem;
  const cudaError_t e = allow_shared(kern, smem, allowed[dev]);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3((unsigned)grid), dim3(kRowsThreads), smem, s, true, p);
}

// Clusters of as many CTAs as the device holds at once beside one another, with two tiles each
// or more.
template <int MODE, int D, int M>
cudaError_t launch_prefill_as(const RowsParams& p, int dev, cudaStream_t s) {
  static std::atomic<int> allowed[kDevices], known[kDevices][kRowsMaxCluster + 1];
  using Lay = RowsLayout<MODE, D, M>;
  const auto kern = rows_prefill_kernel<MODE, D, M>;
  cudaError_t e = allow_shared(kern, Lay::kSmem, allowed[dev]);
  if (e != cudaSuccess) return e;
  const long long units = (long long)p.units_max * p.plan.span.batch * p.plan.hkv;
  constexpr int KT = RowsTile<MODE, D, M>::kKeys;
  const long long tiles = (p.keys_most + KT - 1) / KT + 1;
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

// Units of 16, 32 or 64 rows (fp32 with head_dim 128: up to 32, whose Q in two parts fits).
template <int MODE, int D>
constexpr int rows_most() {
  return MODE == PKV_F32 && D == 128 ? 32 : 64;
}

template <int MODE, int D>
cudaError_t launch_rows_d(const RowsParams& p, bool tree, long long grid, int dev, cudaStream_t s) {
  constexpr int kMost = rows_most<MODE, D>();
  const int rows = p.plan.unit_rows;
  if (tree)
    return rows == 16   ? launch_tree_as<MODE, D, 16>(p, grid, dev, s)
           : rows == 32 ? launch_tree_as<MODE, D, 32>(p, grid, dev, s)
                        : launch_tree_as<MODE, D, kMost>(p, grid, dev, s);
  return rows == 16   ? launch_prefill_as<MODE, D, 16>(p, dev, s)
         : rows == 32 ? launch_prefill_as<MODE, D, 32>(p, dev, s)
                      : launch_prefill_as<MODE, D, kMost>(p, dev, s);
}

template <int MODE, int D>
constexpr int rows_ctas_d(int unit_rows) {
  return unit_rows == 16   ? RowsLayout<MODE, D, 16>::kCtas
         : unit_rows == 32 ? RowsLayout<MODE, D, 32>::kCtas
                           : RowsLayout<MODE, D, rows_most<MODE, D>()>::kCtas;
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
