// Block selection for sparse decode (pkv_select_blocks): a score of every
// block of a query's sequence from its key bounds, and the best of them.
//
// What is computed.  For query token t, kv head g and table entry j, with the
// query coded in 8 bits like the bounds (bounds.cuh):
//   score = max over the G query heads of g of
//           2^(e_q + e_j) * sum_d (q_d >= 0 ? q_d hi_d : q_d lo_d),
// an upper bound of any logit of the block up to the coding of q.  The sum is
// one dot product of length 2 D, [max(q, 0), min(q, 0)] . [hi, lo].  The
// first `sink` and last `recent` entries are taken as they are, the best of
// the others fill the rest; equal scores go to the lower entry.
//
// How.  One cluster of CTAs per (t, g); each CTA scores a contiguous range of
// the entries and keeps the scores in its shared memory, so nothing but the
// result is ever written.  The scores are found on the tensor cores: 16
// blocks by 8 query heads by 16 code bytes per mma, the code bytes c + 128 taken
// as fp16 subnormals (sums of whole numbers up to 255 * 127 * 128 < 2^24, in
// units of 2^-24: exact).  A lane loads 16-byte pieces of its blocks straight
// to registers, and the same pieces of the query, coded once per CTA, from
// shared memory, so the order of k does not matter.
//
// The cut: the scores as ordered integers, counted in 256 bins from the
// cluster-wide range down.  Every CTA counts its own and sums the counts of
// all through distributed shared memory.  Once the bin that holds the cut has
// at most 128 scores (as a rule after the first count), every CTA sends its
// share of those to the others, and each ranks them by (score, entry); a bin
// that stays larger is counted again 8 bits finer, down to equal scores, of
// which the lowest entries are taken.
//
// What bounds it: latency.  One query: a chain of four loads, then with one count
// four cluster barriers and nine block barriers, eleven where scores are ranked:
// 14.9 us for 128 of 8192 blocks (Hkv 8, D 128, G 4), of which the instructions, 2.4 M
// on 64 SMs, are 4.5.  64 queries, 64 of 64 to 513 blocks each, 42 MB of bounds: 16.8 us,
// 4.5 of them instructions at full issue (5.6 M, 34 % of the slots used, 4.4 warps an
// SMSP).  (Scores to a workspace, and the cut in a second launch, took 18 and 23 us.)
#include <climits>
#include <cmath>

#include <cuda_fp16.h>

#include "bounds.cuh"
#include "cluster.cuh"
#include "common.cuh"
#include "mma.cuh"

namespace pkv {
namespace {

constexpr int kSelMaxCluster = 8;
constexpr int kCand = 128;  // scores that are ranked rather than counted
constexpr unsigned kAll = 0xffffffffu;

struct SelectParams {
  const char* q;
  const char* codes;
  const float* scales;
  const int32_t* bt;
  const int32_t* offs;
  const int32_t* tok_seq;
  const int32_t* tok_pos;
  int32_t* sel;
  int32_t* count;
  int* err;
  uint32_t num_blocks;
  int batch, mb, bs, L, layer, hq, hkv, G, K, sink, recent;
  int q_size;  // bytes of an element of q
  int cap;  // scores a CTA can hold
};

// Static shared memory.  What the CTAs of a cluster tell each other they write
// into the others' copies (or add to them) ahead of a cluster barrier, so that
// only the counts of the bins are read across it.
struct SelectShared {
  uint32_t hist[4][256];
  uint32_t range[2];                       // smallest and largest score of the cluster
  uint32_t over0, even0;                   // scores above the cut, and at it, of the CTAs before
  uint32_t cand_n[kSelMaxCluster];         // scores in the cut's bin of each CTA,
  uint32_t cand_key[kSelMaxCluster][kCand];  // themselves,
  uint32_t cand_at[kSelMaxCluster][kCand];   // and their entries
  // not written by others
  uint32_t all_key[kCand], all_at[kCand];
  uint32_t counts[2], ncand, before;
  uint32_t pick[3];
  uint32_t warp_a[32], warp_b[32];
};

// Code bytes b = c + 128 to the fp16 numbers with those bits, the subnormals
// b * 2^-24: two a register, one byte permute each.  The tensor cores take
// subnormals as they are.
__device__ __forceinline__ void codes_as_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("prmt.b32 %0, %1, 0, 0x4140;" : "=r"(lo) : "r"(w));
  asm("prmt.b32 %0, %1, 0, 0x4342;" : "=r"(hi) : "r"(w));
}
constexpr float kUnit = 0x1p-24f, kBias = 128.f * kUnit;

// Order-preserving map of a score to an unsigned integer in [1, 2^32 - 2].
__device__ __forceinline__ uint32_t ordered(float x) {
  uint32_t u = __float_as_uint(x);
  if (u == 0x80000000u) u = 0;  // -0 and +0 are one score
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return min(0xfffffffeu, max(1u, u));
}

// Inclusive sums of (a, b) over the CTA's threads; every thread calls it.
__device__ __forceinline__ void block_scan(uint32_t& a, uint32_t& b, SelectShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(kAll, a, o), y = __shfl_up_sync(kAll, b, o);
    if (lane >= o) { a += x; b += y; }
  }
  if (lane == 31) { sh.warp_a[warp] = a; sh.warp_b[warp] = b; }
  __syncthreads();
  // the warps before this one, one per lane
  a += __reduce_add_sync(kAll, lane < warp ? sh.warp_a[lane] : 0u);
  b += __reduce_add_sync(kAll, lane < warp ? sh.warp_b[lane] : 0u);
  __syncthreads();
}

// Sum of a 32-bit word over the first `n` CTAs of the cluster, four loads in
// flight at a time.
__device__ __forceinline__ uint32_t cluster_sum(uint32_t addr, uint32_t n) {
  uint32_t sum = 0;
  for (uint32_t r = 0; r < n; r += 4) {
    uint32_t v[4];
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u)
      v[u] = r + u < n ? ld_cluster_u32(cluster_map(addr, r + u)) : 0u;
    sum += (v[0] + v[1]) + (v[2] + v[3]);
  }
  return sum;
}

__device__ __forceinline__ uint32_t ld_u32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ void sts_u32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ void sync_all(uint32_t S) {
  if (S > 1)
    cluster_sync();
  else
    __syncthreads();
}

// NT: tiles of 8 query heads.  With one, 80 registers a thread, so that an SM
// holds 24 warps; with two, 12.
template <int D, int NT, int THREADS>
__global__ void __launch_bounds__(THREADS, (NT == 1 ? 768 : 384) / THREADS)
    select_kernel(const SelectParams p) {
  constexpr int LD = D / 64;  // 64-element pieces of a bound
  constexpr int WARPS = THREADS / 32;
  constexpr int QROW = D * 2 + 16;  // bytes of a coded query row, padded against bank conflicts
  constexpr int EPL = D / 32;       // elements of a query row a lane codes
  extern __shared__ uint32_t keys[];
  __shared__ SelectShared sh;
  // the coded query: positive and negative parts, unit * 2^24, bias
  __shared__ __align__(16) unsigned char sq[2][NT * 8 * QROW];
  __shared__ float s_unit[NT * 8], s_bias[NT * 8];
  griddep_wait();
  griddep_launch_dependents();
  uint32_t S;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const uint32_t rank = cluster_rank();
  const int row = blockIdx.x / S;
  const int t = row / p.hkv, g = row - t * p.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const int seq = ld_volatile(p.tok_seq + t), pos = ld_volatile(p.tok_pos + t);
  // this warp's query rows, in flight beside the chain of index loads
  constexpr int QPW = (NT * 8 + WARPS - 1) / WARPS;
  uint32_t qraw[QPW][EPL];
#pragma unroll
  for (int u = 0; u < QPW; ++u) {
    const int h = warp + u * WARPS;
    const char* src = p.q + (((long long)t * p.hq + g * p.G + h) * D + lane * EPL) * p.q_size;
#pragma unroll
    for (int i = 0; i < EPL; ++i) qraw[u][i] = 0;
    if (h < p.G) {
      if (p.q_size == 4) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) qraw[u][i] = ld_u32(src + 4 * i);
      } else {
#pragma unroll
        for (int i = 0; i < EPL / 2; ++i) qraw[u][i] = ld_u32(src + 4 * i);
      }
    }
  }
  int off = 0, n = 0;
  if (seq >= p.batch) {
    if (rank == 0 && tid == 0) set_error(p.err, kErrIndex);
  } else if (seq >= 0) {
    off = p.offs ? p.offs[seq] : 0;
    if (off < 0 || off >= p.bs || pos < 0 || (long long)off + pos >= (long long)p.mb * p.bs) {
      if (rank == 0 && tid == 0) set_error(p.err, kErrCapacity);
    } else {
      n = ((off + pos) >> (31 - __clz(p.bs))) + 1;
    }
  }
  int32_t* out = p.sel + (long long)row * p.K;
  if (rank == 0 && tid == 0) p.count[row] = min(n, p.K);
  if (n <= p.K) {  // all of them, or none (the whole cluster leaves)
    for (int i = rank * THREADS + tid; i < p.K; i += S * THREADS) out[i] = i < n ? i : -1;
    return;
  }
  if (rank == 0) {
    for (int i = tid; i < p.sink; i += THREADS) out[i] = i;
    for (int i = tid; i < p.recent; i += THREADS) out[p.K - p.recent + i] = n - p.recent + i;
  }
  const int need = p.K - p.sink - p.recent;
  if (need == 0) return;
  const int m = n - p.sink - p.recent;  // scored entries, more than need
  const int per = (m + (int)S - 1) / (int)S;
  const int lo = min(m, (int)rank * per), cnt = min(m, lo + per) - lo;

  for (int i = tid; i < 4 * 256; i += THREADS) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) {
    sh.range[0] = 0xffffffffu;
    sh.range[1] = sh.over0 = sh.even0 = sh.counts[0] = sh.counts[1] = sh.ncand = sh.before = 0;
  }
  if (S > 1) cluster_arrive();  // waited for before the first write to another CTA

  // ---- entries of the first tile -------------------------------------------
  const int gl = lane >> 2, qi = lane & 3;
  const int32_t* table = p.bt + (long long)seq * p.mb + p.sink + lo;
  auto entry = [&](int i) { return i < cnt ? ld_volatile(table + i) : -1; };
  constexpr int STEP = WARPS * 16;
  int base = warp * 16;
  int id[2] = {entry(base + gl), entry(base + gl + 8)};

  // ---- the query in 8 bits ---------------------------------------------------
#pragma unroll
  for (int u = 0; u < QPW; ++u) {
    const int h = warp + u * WARPS;
    if (h >= NT * 8) break;
    const uint32_t at = smem_addr(sq[0]) + h * QROW + lane * EPL * 2;
    uint32_t hp[EPL / 2] = {}, hn[EPL / 2] = {};
    int sum = 0;
    float unit = 0.f;
    if (h < p.G) {
      float x[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        x[i] = p.q_size == 4 ? __uint_as_float(qraw[u][i])
               : i & 1       ? bf16_hi(qraw[u][i / 2])
                             : bf16_lo(qraw[u][i / 2]);
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) mx = max(mx, __float_as_uint(x[i]) & 0x7FFFFFFFu);
      mx = __reduce_max_sync(kAll, mx);
      const int e = bound_exponent(mx);
      const float inv = pow2f(-e);
      unit = pow2f(e) * 0x1p24f;
#pragma unroll
      for (int i = 0; i < EPL / 2; ++i) {
        const int a = min(127, max(-127, __float2int_rn(mul_ieee(x[2 * i], inv))));
        const int b = min(127, max(-127, __float2int_rn(mul_ieee(x[2 * i + 1], inv))));
        sum += a + b;
        const __half2 c = __floats2half2_rn((float)a, (float)b);
        const __half2 zero = __half2half2(__ushort_as_half(0));
        const __half2 up = __hmax2(c, zero), down = __hmin2(c, zero);
        hp[i] = *reinterpret_cast<const uint32_t*>(&up);
        hn[i] = *reinterpret_cast<const uint32_t*>(&down);
      }
      sum = __reduce_add_sync(kAll, sum);
    }
#pragma unroll
    for (int i = 0; i < EPL / 2; ++i) {
      sts_u32(at + 4 * i, hp[i]);
      sts_u32(at + NT * 8 * QROW + 4 * i, hn[i]);
    }
    if (lane == 0) {
      s_unit[h] = unit;
      s_bias[h] = -kBias * (float)sum;
    }
  }

  // ---- scores: tiles warp, warp + WARPS, ... of 16 blocks ----------------------
  // rows lane / 4 and + 8 of a tile
  const char* codes0 = p.codes + ((long long)p.layer * p.hkv + g) * (2 * D) + qi * 16;
  const float* scales0 = p.scales + (long long)p.layer * p.hkv + g;
  const uint32_t heads = (uint32_t)p.L * p.hkv;  // of a block
  uint4 w[2][2][LD];
  float unit[2];
  bool ok[2];
  auto load = [&](int at) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ok[r] = (uint32_t)id[r] < p.num_blocks;
      const uint32_t blk = ok[r] ? id[r] : 0u;
      const char* src = codes0 + (unsigned long long)blk * (heads * (2 * D));
#pragma unroll
      for (int side = 0; side < 2; ++side)
#pragma unroll
        for (int k = 0; k < LD; ++k) w[r][side][k] = ld_stream(src + side * D + k * 64);
      unit[r] = scales0[(unsigned long long)blk * heads];
      if (!ok[r] && at + gl + 8 * r < cnt) set_error(p.err, kErrIndex);
      id[r] = entry(at + STEP + gl + 8 * r);  // of the next tile
    }
  };
  if (base < cnt) load(base);
  __syncthreads();
  uint32_t kmin = 0xffffffffu, kmax = 0;
  const uint32_t a_q = smem_addr(sq[0]) + gl * QROW + qi * 32;
  float bias[NT][2], f[NT][2];  // of columns 2 qi, 2 qi + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      bias[nt][c] = s_bias[nt * 8 + 2 * qi + c];
      f[nt][c] = s_unit[nt * 8 + 2 * qi + c];
    }
  const bool second = qi & 1;  // this lane ends up with row gl + 8 instead of gl
#pragma unroll 1
  for (; base < cnt; base += STEP) {
    // Whole numbers (c + 128) q, in units of 2^-24; a dim counts on one side
    // only, so all of a score stays below 2^24 of them.
    float best[2];
    float acc[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[nt][0][c] = bias[nt][c & 1];
        acc[nt][1][c] = 0.f;
      }
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int side = 0; side < 2; ++side)
#pragma unroll
        for (int k = 0; k < LD; ++k) {
          const uint4 &y0 = w[0][side][k], &y1 = w[1][side][k];
          uint32_t a[2][4];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            codes_as_f16(half ? (c ? y0.w : y0.z) : (c ? y0.y : y0.x), a[c][0], a[c][2]);
            codes_as_f16(half ? (c ? y1.w : y1.z) : (c ? y1.y : y1.x), a[c][1], a[c][3]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            // dims k * 64 + qi * 16 + half * 8 .. + 7 of head gl
            const uint4 b = lds128(a_q + (side * NT + nt) * 8 * QROW + k * 128 + half * 16);
            mma16<true>(acc[nt][0], a[0][0], a[0][1], a[0][2], a[0][3], b.x, b.y);
            mma16<true>(acc[nt][1], a[1][0], a[1][1], a[1][2], a[1][3], b.z, b.w);
          }
        }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      best[r] = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float x = (acc[nt][0][2 * r + c] + acc[nt][1][2 * r + c]) * f[nt][c];
          if (nt * 8 + 2 * qi + c < p.G) best[r] = fmaxf(best[r], x);
        }
    }
    const float u = second ? unit[1] : unit[0];
    const bool valid = second ? ok[1] : ok[0];
    if (base + STEP < cnt) load(base + STEP);
    // lanes qi 0 and 2 keep row gl, 1 and 3 row gl + 8
    float mine = second ? best[1] : best[0];
    mine = fmaxf(mine, __shfl_xor_sync(kAll, second ? best[0] : best[1], 1));
    mine = fmaxf(mine, __shfl_xor_sync(kAll, mine, 2));
    const int i = base + gl + (second ? 8 : 0);
    if (i < cnt) {
      const uint32_t key = valid ? ordered(mine * u) : 0u;
      if (qi < 2) keys[i] = key;
      kmin = min(kmin, key);
      kmax = max(kmax, key);
    }
  }

  // ---- the cluster's range of scores ----------------------------------------
  kmin = __reduce_min_sync(kAll, kmin);
  kmax = __reduce_max_sync(kAll, kmax);
  if (lane == 0) { sh.warp_a[warp] = kmin; sh.warp_b[warp] = kmax; }
  if (S > 1) cluster_wait();
  __syncthreads();
  if (warp == 0) {
    kmin = __reduce_min_sync(kAll, lane < WARPS ? sh.warp_a[lane] : 0xffffffffu);
    kmax = __reduce_max_sync(kAll, lane < WARPS ? sh.warp_b[lane] : 0u);
    if (lane < S) {  // one CTA per lane
      const uint32_t a = cluster_map(smem_addr(sh.range), lane);
      red_cluster_min(a, kmin);
      red_cluster_max(a + 4, kmax);
    }
  }
  sync_all(S);
  kmin = sh.range[0];
  kmax = sh.range[1];

  // ---- the cut: 8 bits of (score - smallest) a count ---------------------------
  const uint32_t a_hist = smem_addr(sh.hist);
  uint32_t bits = 32 - __clz(kmax - kmin);
  uint32_t prefix = 0;
  uint32_t left = need;  // to be taken among the scores that match the prefix
  bool ranked = false;   // they are few, and are ranked
#pragma unroll 1
  for (int step = 0; bits > 0; ++step) {
    const uint32_t width = min(8u, bits), shift = bits - width, mask = (1u << width) - 1;
    for (int i = tid; i < cnt; i += THREADS) {
      const uint32_t x = keys[i] - kmin;
      if ((bits < 32 ? x >> bits : 0u) == prefix) atomicAdd(&sh.hist[step][(x >> shift) & mask], 1u);
    }
    sync_all(S);
    // a thread sums its bins over the CTAs; the scan runs from the top bin down
    constexpr int BPT = (256 + THREADS - 1) / THREADS;
    uint32_t c[BPT], sum = 0, dummy = 0;
#pragma unroll
    for (int u = 0; u < BPT; ++u) {
      const int bin = 255 - (tid * BPT + u);
      c[u] = bin >= 0 ? cluster_sum(a_hist + (step * 256 + bin) * 4, S) : 0u;
      sum += c[u];
    }
    uint32_t above = sum;
    block_scan(above, dummy, sh);
    above -= sum;
#pragma unroll
    for (int u = 0; u < BPT; ++u) {
      if (above < left && above + c[u] >= left) {
        sh.pick[0] = 255 - (tid * BPT + u);
        sh.pick[1] = left - above;
        sh.pick[2] = c[u];
      }
      above += c[u];
    }
    __syncthreads();
    prefix = (prefix << width) | sh.pick[0];
    left = sh.pick[1];
    const uint32_t found = sh.pick[2];
    bits = shift;
    __syncthreads();
    if (left == found) break;  // every score of the bin is taken
    if (bits > 0 && found <= kCand) {
      ranked = true;
      break;
    }
  }
  // keys from here on lie above the bin of the cut (no key is 2^32 - 1)
  const unsigned long long next = kmin + ((prefix + 1ull) << bits);
  const uint32_t limit = next > 0xffffffffull ? 0xffffffffu : (uint32_t)next;

  // ---- counts above the cut, and at it; the few that are ranked -----------------
  uint32_t over = 0, even = 0;
  for (int i = tid; i < cnt; i += THREADS) {
    const uint32_t key = keys[i];
    over += key >= limit;
    if (key < limit && (key - kmin) >> bits == prefix) {
      ++even;
      if (ranked) {
        const uint32_t slot = atomicAdd(&sh.ncand, 1u);
        for (uint32_t r = 0; r < S; ++r) {
          st_cluster_u32(cluster_map(smem_addr(&sh.cand_key[rank][slot]), r), key);
          st_cluster_u32(cluster_map(smem_addr(&sh.cand_at[rank][slot]), r), lo + i);
        }
      }
    }
  }
  over = __reduce_add_sync(kAll, over);
  even = __reduce_add_sync(kAll, even);
  if (lane == 0) {
    atomicAdd(&sh.counts[0], over);
    atomicAdd(&sh.counts[1], even);
  }
  __syncthreads();
  if (tid < S) {
    if (tid > rank) {
      red_cluster_add(cluster_map(smem_addr(&sh.over0), tid), sh.counts[0]);
      red_cluster_add(cluster_map(smem_addr(&sh.even0), tid), sh.counts[1]);
    }
    st_cluster_u32(cluster_map(smem_addr(&sh.cand_n[rank]), tid), sh.ncand);
  }
  sync_all(S);  // the last word from another CTA
  const uint32_t even0 = sh.even0;
  uint32_t before = sh.over0;
  if (ranked) {
    // put the bin's scores of all CTAs in one list, rank them, and mark the taken
    // ones among this CTA's with a key above the limit, the others with one below
    const uint32_t nr = lane < S ? sh.cand_n[lane] : 0u;
    uint32_t start = nr;  // of the scores of CTA `lane`
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, start, o);
      if (lane >= o) start += y;
    }
    const uint32_t at = __shfl_sync(kAll, start, 31);
    start -= nr;
    for (uint32_t r = warp; r < S; r += WARPS) {
      const uint32_t n0 = __shfl_sync(kAll, nr, r), s0 = __shfl_sync(kAll, start, r);
      for (uint32_t i = lane; i < n0; i += 32) {
        sh.all_key[s0 + i] = sh.cand_key[r][i];
        sh.all_at[s0 + i] = sh.cand_at[r][i];
      }
    }
    __syncthreads();
    for (uint32_t i = warp; i < at; i += WARPS) {
      const uint32_t key = sh.all_key[i], e = sh.all_at[i];
      uint32_t better = 0;
      for (uint32_t j = lane; j < at; j += 32) {
        const uint32_t k2 = sh.all_key[j];
        better += k2 > key || (k2 == key && sh.all_at[j] < e);
      }
      const bool taken = __reduce_add_sync(kAll, better) < left;
      if (lane == 0) {
        if ((int)e >= lo && (int)e < lo + cnt) keys[e - lo] = taken ? 0xffffffffu : 0u;
        if (taken && (int)e < lo) atomicAdd(&sh.before, 1u);
      }
    }
    __syncthreads();
    before += sh.before;
    left = 0;  // none is taken for its place any more
  }

  // ---- write the taken entries in order: a thread's are consecutive --------------
  const int seg = (cnt + THREADS - 1) / THREADS;
  const int i0 = min(cnt, tid * seg), i1 = min(cnt, i0 + seg);
  over = even = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t key = keys[i];
    over += key >= limit;
    even += left > 0 && key < limit && (key - kmin) >> bits == prefix;
  }
  const uint32_t my_over = over, my_even = even;
  block_scan(over, even, sh);
  over += before - my_over;
  even += even0 - my_even;
  for (int i = i0; i < i1; ++i) {
    const uint32_t key = keys[i];
    const bool ov = key >= limit;
    const bool eq = left > 0 && !ov && (key - kmin) >> bits == prefix;
    if (ov || (eq && even < left)) out[p.sink + over + min(even, left)] = p.sink + lo + i;
    over += ov;
    even += eq;
  }
}

constexpr int kSelMaxCap = 40 * 1024;  // scores of one CTA: 160 KB

// Threads T of a CTA and CTAs S of a cluster.  A warp's time for a tile of 16
// blocks grows slowly with the L warps on its SM, about as 64 + L, and the cut
// costs it that of 4 tiles, in a cluster of one and a quarter for each CTA more.
// The pair with the least
//     rounds * (tiles of a warp + 4 + 1 + S / 4) * (64 + L)
// is taken; clusters only where one round of them is enough, unless the scores
// need their room.  Of 284 cases timed with every pair (1 to 1000 rows of 90 to
// 8000 blocks, D 64 and 128, G 4 and 16) it is within 14 % of the best one in all
// and within 10 % in 280.  T x S for D 128, G 4: 43 rows of 2000 blocks 384 x 3 12.5
// us, 384 x 7 19.7, 768 x 1 15.8; 170 rows of 2000 192 x 3 24.1, 384 x 1 26.3, 192 x 1
// 32.6; 8 of 8000 768 x 8 13.8, 384 x 8 15.2.
template <int D, int NT>
cudaError_t launch_select(SelectParams& p, unsigned rows, int dev, int sms, cudaStream_t s) {
  // (768 threads have no registers for a second set of sums)
  constexpr int kThreads[2][3] = {{768, 384, 192}, {384, 192, 0}}, kChoices = 4 - NT;
  constexpr int kPart = kSelMaxCap * 4 / 8;  // bytes: shared memory is asked for in eighths
  static std::atomic<int> allowed[kDevices][3], known[kDevices][3][9][kSelMaxCluster + 1];
  void (*const kern[3])(SelectParams) = {
      NT == 1 ? select_kernel<D, 1, 768> : select_kernel<D, 2, 384>,
      NT == 1 ? select_kernel<D, 1, 384> : select_kernel<D, 2, 192>,
      NT == 1 ? select_kernel<D, 1, 192> : nullptr};
  const int tiles = (p.mb + 15) / 16;
  int choice = -1, ctas = 1;
  long long least = LLONG_MAX;
  for (int c = 0; c < kChoices; ++c) {
    const int T = kThreads[NT - 1][c], W = T / 32;
    cudaError_t e = allow_shared(kern[c], kSelMaxCap * 4, allowed[dev][c]);
    if (e != cudaSuccess) return e;
    for (int S = 1; S <= kSelMaxCluster && (S - 1) * W < tiles; ++S) {
      const int cap = (p.mb + S - 1) / S, part = (cap * 4 + kPart - 1) / kPart;
      if (cap > kSelMaxCap) continue;
      int fit = 0;
      e = clusters_held(kern[c], T, (size_t)part * kPart, (unsigned)S, known[dev][c][part][S], &fit);
      if (e != cudaSuccess) return e;
      if (fit < 1) break;
      const long long rounds = (rows + (long long)fit - 1) / fit;
      // (a sixteenth stays free: 96 rows of 1600 blocks take 18.5 us as 384 x 3, of which
      // 97 fit, 14.7 as 768 x 1)
      const bool one_round = rows + rows / 16 <= (unsigned)fit;
      if (S > 1 && !one_round && (p.mb + S - 2) / (S - 1) <= kSelMaxCap) break;
      const long long held = rounds > 1 ? (long long)fit * S : (long long)rows * S;
      const long long L = W * ((held + sms - 1) / sms);
      const long long each = (tiles + W * S - 1) / (W * S);  // tiles of a warp
      const long long cost = rounds * (4 * each + 16 + (S > 1 ? 4 + S : 0)) * (64 + L);
      if (cost < least) {
        least = cost;
        choice = c;
        ctas = S;
      }
    }
  }
  if (choice < 0) return cudaErrorInvalidConfiguration;
  p.cap = (p.mb + ctas - 1) / ctas;
  return launch_clusters(kern[choice], dim3(rows * (unsigned)ctas), dim3(kThreads[NT - 1][choice]),
                         (size_t)p.cap * 4, (unsigned)ctas, s, p);
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_select_blocks(const pkv_pool* pool, int32_t layer,
                                        const void* bound_codes, const float* bound_scales,
                                        const void* q, int32_t num_q_heads,
                                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                                        const int32_t* offsets, int32_t batch,
                                        const int32_t* token_seq, const int32_t* token_pos,
                                        int32_t num_tokens, int32_t num_selected, int32_t sink,
                                        int32_t recent, int32_t* selected,
                                        int32_t* selected_count, cudaStream_t stream) {
  pkv::PoolView v;
  int st = pkv::pool_view(pool, false, &v);
  if (st != PKV_OK) return (pkv_status)st;
  if (layer < 0 || layer >= v.num_layers || batch < 0 || num_tokens < 0 || num_q_heads <= 0 ||
      num_selected <= 0 || sink < 0 || recent < 0 ||
      (int64_t)sink + recent > num_selected || num_q_heads % v.num_kv_heads != 0)
    return PKV_ERR_INVALID_ARG;
  const int G = num_q_heads / v.num_kv_heads;
  if ((v.head_dim != 64 && v.head_dim != 128) || G > 16) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!bound_codes || !bound_scales || !q || !token_seq || !token_pos || !selected ||
      !selected_count || (batch > 0 && (!block_tables || max_blocks_per_seq <= 0)))
    return PKV_ERR_INVALID_ARG;
  if (!pkv::aligned(bound_codes, 16) || !pkv::aligned(bound_scales, 4) || !pkv::aligned(q, 16) ||
      !pkv::aligned(block_tables, 4) || !pkv::aligned(offsets, 4) ||
      !pkv::aligned(token_seq, 4) || !pkv::aligned(token_pos, 4) || !pkv::aligned(selected, 4) ||
      !pkv::aligned(selected_count, 4))
    return PKV_ERR_INVALID_ARG;
  const int mb = batch > 0 ? max_blocks_per_seq : 1;
  // table positions are 32-bit in the kernel, and a cluster holds every score of a row
  if ((int64_t)mb * v.block_size > INT32_MAX || mb > pkv::kSelMaxCluster * pkv::kSelMaxCap)
    return PKV_ERR_UNSUPPORTED;
  if ((int64_t)v.num_layers * v.num_kv_heads * 2 * v.head_dim > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)num_tokens * v.num_kv_heads;
  if (rows > INT32_MAX / pkv::kSelMaxCluster) return PKV_ERR_UNSUPPORTED;
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
  pkv::SelectParams p;
  p.q = static_cast<const char*>(q);
  p.codes = static_cast<const char*>(bound_codes);
  p.scales = bound_scales;
  p.bt = block_tables;
  p.offs = offsets;
  p.tok_seq = token_seq;
  p.tok_pos = token_pos;
  p.sel = selected;
  p.count = selected_count;
  p.err = err;
  p.num_blocks = (uint32_t)(v.num_blocks < INT32_MAX ? v.num_blocks : INT32_MAX);
  p.batch = batch;
  p.mb = mb;
  p.bs = v.block_size;
  p.L = v.num_layers;
  p.layer = layer;
  p.hq = num_q_heads;
  p.hkv = v.num_kv_heads;
  p.G = G;
  p.K = num_selected;
  p.sink = sink;
  p.recent = recent;
  p.q_size = v.io_size;
  const unsigned r = (unsigned)rows;
  cudaError_t e;
  if (v.head_dim == 64)
    e = G <= 8 ? pkv::launch_select<64, 1>(p, r, dev, sms, stream)
               : pkv::launch_select<64, 2>(p, r, dev, sms, stream);
  else
    e = G <= 8 ? pkv::launch_select<128, 1>(p, r, dev, sms, stream)
               : pkv::launch_select<128, 2>(p, r, dev, sms, stream);
  if ((st = pkv::launch_status(e)) != PKV_OK) return (pkv_status)st;
  return validate ? (pkv_status)pkv::read_and_clear_error_word(err, stream) : PKV_OK;
}
