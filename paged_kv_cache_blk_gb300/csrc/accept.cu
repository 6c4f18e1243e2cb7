// Accepted drafted tokens moved right behind the context (pkv_accept_tokens).
//
// What is done.  The n drafted tokens of a sequence sit at positions ctx .. ctx + n - 1;
// the accepted ones a_0 < a_1 < ... are to follow the context as a verified chain would:
// the K and V rows of position ctx + a_k go to position ctx + k, in one layer or in all.
//
// What bounds it: each moved row once in and once out, and for a user or two the chain of
// loads (sequence, path, table entry, row).
//
// How.  A CTA per (sequence, layer, K or V) first turns the path into rows of the pool;
// then each thread owns 16-byte columns of the row and takes the path's tokens in order,
// kBatch loads before their stores.  a_k >= k and ascending, so a store never overwrites a
// row that a later token still has to read, and as only this thread touches its columns
// no barrier stands between tokens.  5 rows of 32 layers: 3.2 us on the device, of a call's
// 7.5; up to 8 rows of each of 64 sequences in 16 layers, whose bytes take 2.3 us, 6.2 (one call
// after another, replayed).
#include <climits>

#include "common.cuh"
#include "span.cuh"

namespace pkv {
namespace {

constexpr int kAcceptThreads = 128;
constexpr int kBatch = 8;     // rows in flight a thread
constexpr int kPathMost = 1024;  // entries of a path turned into rows at a time

struct AcceptParams {
  SpanParams span;
  char* k;
  char* v;
  const int32_t* bt;
  const int32_t* path;
  const int32_t* count;
  int* err;
  long long num_blocks;
  int path_most, L, first_layer, row_bytes, bs_bits;
  int check_only;  // validate mode: nothing is moved
};

// (stays before the stores that follow it)
__device__ __forceinline__ uint4 ld_row(const char* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptParams p) {
  __shared__ long long src[kPathMost], dst[kPathMost];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x, layer = p.first_layer + (int)(blockIdx.y >> 1);
  char* cache = blockIdx.y & 1 ? p.v : p.k;
  const bool report = blockIdx.y == 0 && threadIdx.x == 0;
  const SeqSpan s = seq_span(p.span, b);
  if (s.bad && report) set_error(p.err, kErrCapacity);
  const int count = s.ok ? p.count[b] : 0;
  if (count == 0) return;
  const int32_t* path = p.path + (long long)b * p.path_most;
  const int32_t* table = p.bt + (long long)b * p.span.mb;
  // the whole path first: a path that does not ascend within the drafted tokens, or names a
  // block outside the pool, moves nothing
  bool bad = count < 0 || count > p.path_most || count > s.n;
  int what = bad ? kErrCapacity : 0;
  if (!bad) {
    const int pos0 = s.off + s.ctx;
    for (int i = threadIdx.x; i < count; i += kAcceptThreads) {
      const int a = path[i];
      if (a < i || a >= s.n || (i > 0 && path[i - 1] >= a)) {
        what |= kErrIndex;
        continue;
      }
      if (a == i) continue;
      const int from = table[(pos0 + a) >> p.bs_bits], to = table[(pos0 + i) >> p.bs_bits];
      if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks) what |= kErrIndex;
    }
  }
  what = __syncthreads_or(what);
  if (what) {
    if (report) set_error(p.err, bad ? kErrCapacity : kErrIndex);
    return;
  }
  if (p.check_only) return;
  const int chunks = p.row_bytes >> 4, pos0 = s.off + s.ctx;
  auto row_of = [&](int pos) {
    const long long blk = table[pos >> p.bs_bits];
    return (((blk * p.L + layer) << p.bs_bits) + (pos & ((1 << p.bs_bits) - 1))) * p.row_bytes;
  };
  for (int i0 = 0; i0 < count; i0 += kPathMost) {
    const int m = min(kPathMost, count - i0);
    __syncthreads();
    for (int i = threadIdx.x; i < m; i += kAcceptThreads) {
      const int a = path[i0 + i];
      src[i] = a == i0 + i ? -1 : row_of(pos0 + a);  // -1: it is where it belongs
      dst[i] = a == i0 + i ? -1 : row_of(pos0 + i0 + i);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < chunks; c += kAcceptThreads) {
      for (int i = 0; i < m; i += kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (i + u < m && src[i + u] >= 0)
            x[u] = ld_row(cache + src[i + u] + c * 16ll);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (i + u < m && src[i + u] >= 0) st_global(cache + dst[i + u] + c * 16ll, x[u]);
      }
    }
  }
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_accept_tokens(const pkv_pool* pool, int32_t layer,
                                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                                        const int32_t* seq_lens, const int32_t* offsets,
                                        const int64_t* cu_q, int32_t batch,
                                        const int32_t* accepted,
                                        int32_t max_accepted, const int32_t* accepted_count,
                                        cudaStream_t stream) {
  pkv::PoolView v;
  int st = pkv::pool_view(pool, true, &v);
  if (st != PKV_OK) return (pkv_status)st;
  if (layer < -1 || layer >= v.num_layers || batch < 0 || max_accepted < 0)
    return PKV_ERR_INVALID_ARG;
  if (batch == 0 || max_accepted == 0) return PKV_OK;
  if (!block_tables || !seq_lens || !cu_q || !accepted || !accepted_count ||
      max_blocks_per_seq <= 0)
    return PKV_ERR_INVALID_ARG;
  if (!pkv::aligned(block_tables, 4) || !pkv::aligned(seq_lens, 4) || !pkv::aligned(offsets, 4) ||
      !pkv::aligned(cu_q, 8) || !pkv::aligned(accepted, 4) || !pkv::aligned(accepted_count, 4))
    return PKV_ERR_INVALID_ARG;
  const int layers = layer < 0 ? v.num_layers : 1;
  // positions and the grid are 32-bit in the kernel
  if ((int64_t)max_blocks_per_seq * v.block_size > pkv::kMaxPositions || layers > 32767)
    return PKV_ERR_UNSUPPORTED;
  int optin, grid, validate;
  int* err;
  if ((st = pkv::device_facts(&optin, &err, &grid, &validate)) != PKV_OK) return (pkv_status)st;
  pkv::AcceptParams p = {};
  p.span.lens = seq_lens;
  p.span.offs = offsets;
  p.span.cu_q = reinterpret_cast<const long long*>(cu_q);
  p.span.total_q = LLONG_MAX;
  p.span.batch = batch;
  p.span.mb = max_blocks_per_seq;
  p.span.bs = v.block_size;
  p.span.max_q_len = INT_MAX;
  p.k = v.k_mut;
  p.v = v.v_mut;
  p.bt = block_tables;
  p.path = accepted;
  p.count = accepted_count;
  p.err = err;
  p.num_blocks = v.num_blocks;
  p.path_most = max_accepted;
  p.L = v.num_layers;
  p.first_layer = layer < 0 ? 0 : layer;
  p.row_bytes = v.row_bytes;
  while (1 << p.bs_bits < v.block_size) ++p.bs_bits;
  if (validate) {
    p.check_only = 1;
    if ((st = pkv::clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
    if ((st = pkv::launch_status(pkv::launch_kernel(pkv::accept_kernel, dim3((unsigned)batch),
                                                    dim3(pkv::kAcceptThreads), 0, stream, true,
                                                    p))) != PKV_OK)
      return (pkv_status)st;
    if ((st = pkv::read_and_clear_error_word(err, stream)) != PKV_OK) return (pkv_status)st;
    p.check_only = 0;
  }
  st = pkv::launch_status(pkv::launch_kernel(pkv::accept_kernel,
                                             dim3((unsigned)batch, (unsigned)(2 * layers)),
                                             dim3(pkv::kAcceptThreads), 0, stream, true, p));
  if (st != PKV_OK) return (pkv_status)st;
  return validate ? (pkv_status)pkv::read_and_clear_error_word(err, stream) : PKV_OK;
}
