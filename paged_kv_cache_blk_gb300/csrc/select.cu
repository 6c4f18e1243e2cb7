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
// blocks by 8 query heads by 16 code bytes per mma, the codes turned to fp16
// whole numbers in registers (products and sums below 2^24: exact).  A lane
// loads 16-byte pieces of its two blocks straight to registers; with the same
// pieces of the query in its B fragments, the order of k does not matter.
// The cut is a radix search over the scores as ordered integers, from their
// cluster-wide range down, 8 bits a step: every CTA counts its own scores and
// sums the counts of all through distributed shared memory.
#include <cmath>

#include <cuda_fp16.h>

#include "bounds.cuh"
#include "cluster.cuh"
#include "common.cuh"

namespace pkv {
namespace {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
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
  long long num_blocks;
  int batch, mb, bs, L, layer, hq, hkv, G, K, sink, recent;
  int cap;  // scores a CTA can hold
};

// Static shared memory: what the CTAs of a cluster read of each other.
struct SelectShared {
  uint32_t hist[4][256];
  uint32_t range[2];  // smallest and largest score of this CTA
  uint32_t counts[2];
  uint32_t warp_a[kSelWarps], warp_b[kSelWarps];
  uint32_t total[256];
  uint32_t pick[3];
};

__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  // bytes c + 128 -> fp16 1024 + byte -> minus 1152
  uint32_t a, b;
  asm("prmt.b32 %0, %1, 0x64646464, 0x4140;" : "=r"(a) : "r"(w));
  asm("prmt.b32 %0, %1, 0x64646464, 0x4342;" : "=r"(b) : "r"(w));
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Order-preserving map of a score to an unsigned integer, at least 1.
__device__ __forceinline__ uint32_t ordered(float x) {
  uint32_t u = __float_as_uint(x);
  if (u == 0x80000000u) u = 0;  // -0 and +0 are one score
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return u ? u : 1u;
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
  for (int w = 0; w < warp; ++w) { a += sh.warp_a[w]; b += sh.warp_b[w]; }
  __syncthreads();
}

// T: type of q; NT: tiles of 8 query heads.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
  constexpr int LD = D / 64;  // 16-byte pieces of one bound that a lane holds
  extern __shared__ uint32_t keys[];
  __shared__ SelectShared sh;
  griddep_wait();
  griddep_launch_dependents();
  uint32_t S;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const uint32_t rank = cluster_rank();
  const int row = blockIdx.x / S;
  const int t = row / p.hkv, g = row - t * p.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const int seq = p.tok_seq[t], pos = p.tok_pos[t];
  int off = 0, n = 0;
  if (seq >= p.batch) {
    if (rank == 0 && tid == 0) set_error(p.err, kErrIndex);
  } else if (seq >= 0) {
    off = p.offs ? p.offs[seq] : 0;
    if (off < 0 || off >= p.bs || pos < 0 || (long long)off + pos >= (long long)p.mb * p.bs) {
      if (rank == 0 && tid == 0) set_error(p.err, kErrCapacity);
    } else {
      n = (off + pos) / p.bs + 1;
    }
  }
  int32_t* out = p.sel + (long long)row * p.K;
  if (rank == 0 && tid == 0) p.count[row] = min(n, p.K);
  if (n <= p.K) {  // all of them, or none (the whole cluster leaves)
    for (int i = rank * kSelThreads + tid; i < p.K; i += S * kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  if (rank == 0) {
    for (int i = tid; i < p.sink; i += kSelThreads) out[i] = i;
    for (int i = tid; i < p.recent; i += kSelThreads) out[p.K - p.recent + i] = n - p.recent + i;
  }
  int need = p.K - p.sink - p.recent;
  if (need == 0) return;
  const int m = n - p.sink - p.recent;  // scored entries, more than need
  const int per = (m + (int)S - 1) / (int)S;
  const int lo = min(m, (int)rank * per), cnt = min(m, lo + per) - lo;

  // ---- the query: 8-bit codes as fp16 B fragments ------------------------
  const int gl = lane >> 2, qi = lane & 3;
  uint32_t bp[NT][LD][4][2], bn[NT][LD][4][2];  // positive and negative parts
  float f0[NT], f1[NT];                         // 2^e_q of columns 2 qi, 2 qi + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int h = nt * 8 + gl;
    float x[LD][16];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const char* src = p.q + (((long long)t * p.hq + g * p.G + h) * D + i * 64 + qi * 16) *
                                  (long long)sizeof(T);
#pragma unroll
      for (int v = 0; v < (int)sizeof(T); ++v) {
        const uint4 r = h < p.G ? *reinterpret_cast<const uint4*>(src + 16 * v)
                                : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (sizeof(T) == 2) {
            x[i][8 * v + 2 * k] = bf16_lo(w[k]);
            x[i][8 * v + 2 * k + 1] = bf16_hi(w[k]);
          } else {
            x[i][4 * v + k] = __uint_as_float(w[k]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) mx = max(mx, __float_as_uint(x[i][k]) & 0x7FFFFFFFu);
    }
    mx = max(mx, __shfl_xor_sync(kAll, mx, 1));
    mx = max(mx, __shfl_xor_sync(kAll, mx, 2));
    const int e = bound_exponent(mx);
    const float inv = pow2f(-e);
#pragma unroll
    for (int i = 0; i < LD; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int a = min(127, max(-127, __float2int_rn(mul_ieee(x[i][2 * k], inv))));
        const int b = min(127, max(-127, __float2int_rn(mul_ieee(x[i][2 * k + 1], inv))));
        const __half2 hp = __floats2half2_rn((float)max(a, 0), (float)max(b, 0));
        const __half2 hn = __floats2half2_rn((float)min(a, 0), (float)min(b, 0));
        bp[nt][i][k >> 1][k & 1] = *reinterpret_cast<const uint32_t*>(&hp);
        bn[nt][i][k >> 1][k & 1] = *reinterpret_cast<const uint32_t*>(&hn);
      }
    const float unit = pow2f(e);
    f0[nt] = __shfl_sync(kAll, unit, 8 * qi);
    f1[nt] = __shfl_sync(kAll, unit, 8 * qi + 4);
  }

  // ---- scores --------------------------------------------------------------
  uint32_t kmin = 0xffffffffu, kmax = 0;
  const int32_t* table = p.bt + (long long)seq * p.mb + p.sink + lo;
  for (int base = warp * 16; base < cnt; base += kSelWarps * 16) {
    uint4 w[2][2][LD];
    float unit[2];
    bool ok[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = base + gl + 8 * r;
      const int blk = i < cnt ? table[i] : -1;
      ok[r] = blk >= 0 && blk < p.num_blocks;
      if (i < cnt && !ok[r] && qi == 0) set_error(p.err, kErrIndex);
      const long long head = ((long long)(ok[r] ? blk : 0) * p.L + p.layer) * p.hkv + g;
      const char* src = p.codes + head * (2 * D) + qi * 16;
#pragma unroll
      for (int side = 0; side < 2; ++side)
#pragma unroll
        for (int k = 0; k < LD; ++k) w[r][side][k] = ld_stream(src + side * D + k * 64);
      unit[r] = p.scales[head];
    }
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[nt][c] = 0.f;
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
      for (int k = 0; k < LD; ++k) {
        const uint32_t u0[4] = {w[0][side][k].x, w[0][side][k].y, w[0][side][k].z, w[0][side][k].w};
        const uint32_t u1[4] = {w[1][side][k].x, w[1][side][k].y, w[1][side][k].z, w[1][side][k].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t a0, a1, a2, a3;
          codes_to_f16(u0[c], a0, a2);
          codes_to_f16(u1[c], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(acc[nt], a0, a1, a2, a3, side ? bn[nt][k][c][0] : bp[nt][k][c][0],
                    side ? bn[nt][k][c][1] : bp[nt][k][c][1]);
        }
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float best = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt * 8 + 2 * qi < p.G) best = fmaxf(best, acc[nt][2 * r] * f0[nt]);
        if (nt * 8 + 2 * qi + 1 < p.G) best = fmaxf(best, acc[nt][2 * r + 1] * f1[nt]);
      }
      best = fmaxf(best, __shfl_xor_sync(kAll, best, 1));
      best = fmaxf(best, __shfl_xor_sync(kAll, best, 2));
      const int i = base + gl + 8 * r;
      if (i < cnt) {
        const uint32_t key = ok[r] ? ordered(best * unit[r]) : 0u;
        if (qi == 0) keys[i] = key;
        kmin = min(kmin, key);
        kmax = max(kmax, key);
      }
    }
  }

  // ---- the cluster's range of scores ----------------------------------------
  kmin = __reduce_min_sync(kAll, kmin);
  kmax = __reduce_max_sync(kAll, kmax);
  if (lane == 0) { sh.warp_a[warp] = kmin; sh.warp_b[warp] = kmax; }
  for (int i = tid; i < 4 * 256; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kSelWarps; ++w) {
      kmin = min(kmin, sh.warp_a[w]);
      kmax = max(kmax, sh.warp_b[w]);
    }
    sh.range[0] = kmin;
    sh.range[1] = kmax;
  }
  cluster_sync();
  const uint32_t a_range = smem_addr(sh.range), a_hist = smem_addr(sh.hist),
                 a_counts = smem_addr(sh.counts);
  for (uint32_t r = 0; r < S; ++r) {
    const uint32_t a = cluster_map(a_range, r);
    kmin = min(kmin, ld_cluster_u32(a));
    kmax = max(kmax, ld_cluster_u32(a + 4));
  }

  // ---- the cut: 8 bits of (score - smallest) a step ---------------------------
  uint32_t bits = 32 - __clz(kmax - kmin);
  uint32_t prefix = 0;
  uint32_t left = need;  // to be taken among the scores that match the prefix
#pragma unroll 1
  for (int step = 0; bits > 0; ++step) {
    const uint32_t width = min(8u, bits), shift = bits - width, mask = (1u << width) - 1;
    for (int i = tid; i < cnt; i += kSelThreads) {
      const uint32_t x = keys[i] - kmin;
      if ((bits < 32 ? x >> bits : 0u) == prefix) atomicAdd(&sh.hist[step][(x >> shift) & mask], 1u);
    }
    cluster_sync();
    // thread b sums bin 255 - b over the CTAs, so the scan runs from the top
    const int bin = 255 - tid;
    uint32_t c = 0;
    for (uint32_t r = 0; r < S; ++r)
      c += ld_cluster_u32(cluster_map(a_hist + (step * 256 + bin) * 4, r));
    uint32_t above = c, dummy = 0;
    block_scan(above, dummy, sh);
    if (above >= left && above - c < left) {
      sh.pick[0] = bin;
      sh.pick[1] = left - (above - c);
      sh.pick[2] = c;
    }
    __syncthreads();
    prefix = (prefix << width) | sh.pick[0];
    left = sh.pick[1];
    const bool whole = left == sh.pick[2];  // every score of the bin is taken
    bits = shift;
    __syncthreads();
    if (whole) break;
  }

  // ---- write the taken entries in order ---------------------------------------
  // a thread's entries are consecutive; `over` are above the cut, `even` match it
  const int seg = (cnt + kSelThreads - 1) / kSelThreads;
  const int i0 = min(cnt, tid * seg), i1 = min(cnt, i0 + seg);
  uint32_t over = 0, even = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t x = (keys[i] - kmin) >> bits;
    over += x > prefix;
    even += x == prefix;
  }
  const uint32_t my_over = over, my_even = even;
  block_scan(over, even, sh);
  if (tid == kSelThreads - 1) { sh.counts[0] = over; sh.counts[1] = even; }
  over -= my_over;
  even -= my_even;
  cluster_sync();
  for (uint32_t r = 0; r < rank; ++r) {
    const uint32_t a = cluster_map(a_counts, r);
    over += ld_cluster_u32(a);
    even += ld_cluster_u32(a + 4);
  }
  for (int i = i0; i < i1; ++i) {
    const uint32_t x = (keys[i] - kmin) >> bits;
    const bool eq = x == prefix;
    if (x > prefix || (eq && even < left)) out[p.sink + over + min(even, left)] = p.sink + lo + i;
    over += x > prefix;
    even += eq;
  }
  cluster_sync();  // no CTA leaves while another may still read its counts
}

template <typename T, int D>
cudaError_t launch_select_d(const SelectParams& p, unsigned grid, unsigned S, cudaStream_t s) {
  const size_t smem = (size_t)p.cap * 4;
  if (p.G <= 8)
    return launch_clusters(select_kernel<T, D, 1>, dim3(grid), dim3(kSelThreads), smem, S, s, p);
  return launch_clusters(select_kernel<T, D, 2>, dim3(grid), dim3(kSelThreads), smem, S, s, p);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int kSelMaxCluster = 8;
constexpr int kSelMaxCap = 40 * 1024;  // scores of one CTA: 160 KB

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
  const int64_t rows = (int64_t)num_tokens * v.num_kv_heads;
  if (rows > INT32_MAX / pkv::kSelMaxCluster) return PKV_ERR_UNSUPPORTED;
  int optin, grid, validate, sms;
  int* err;
  if ((st = pkv::device_facts(&optin, &err, &grid, &validate)) != PKV_OK) return (pkv_status)st;
  if ((st = pkv::device_sm_count(&sms)) != PKV_OK) return (pkv_status)st;
  if (validate) {
    if ((st = pkv::clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
    if ((st = pkv::launch_status(pkv::launch_validate_tokens(
             v, block_tables, mb, offsets, batch, token_seq, token_pos, num_tokens, err,
             stream))) != PKV_OK)
      return (pkv_status)st;
    if ((st = pkv::read_and_clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
  }
  // CTAs of a cluster: until two per SM are there, each with 128 entries or
  // more, and as many as the scores need room.
  unsigned S = 1;
  while ((int)S < pkv::kSelMaxCluster &&
         ((rows * S < 2 * sms && mb / S > 128) || (mb + S - 1) / S > pkv::kSelMaxCap))
    S *= 2;
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
  p.num_blocks = v.num_blocks;
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
  p.cap = (mb + (int)S - 1) / (int)S;
  const unsigned ctas = (unsigned)rows * S;
  cudaError_t e;
  if (v.io_size == 2)
    e = v.head_dim == 64 ? pkv::launch_select_d<__nv_bfloat16, 64>(p, ctas, S, stream)
                         : pkv::launch_select_d<__nv_bfloat16, 128>(p, ctas, S, stream);
  else
    e = v.head_dim == 64 ? pkv::launch_select_d<float, 64>(p, ctas, S, stream)
                         : pkv::launch_select_d<float, 128>(p, ctas, S, stream);
  if ((st = pkv::launch_status(e)) != PKV_OK) return (pkv_status)st;
  return validate ? (pkv_status)pkv::read_and_clear_error_word(err, stream) : PKV_OK;
}
