// The index step on the device: (sequence, position) -> slot through the
// block tables, and the byte offset of a token row; shared by the slot mapping
// and the scatters (copy_kernels.cu, rope.cu).
#pragma once

#include <cstdint>

#include "common.cuh"

namespace pkv {

// Byte offset of row j of block `blk` in layer `layer`.
__device__ __forceinline__ long long row_offset(long long blk, int layer, int j, int L, int bs,
                                                int row_bytes) {
  return ((blk * L + layer) * (long long)bs + j) * (long long)row_bytes;
}

// Where the slots of a scatter come from: read from slot_mapping, or (the
// fused append) computed from (sequence, position) pairs through the tables.
struct SlotSrc {
  const int64_t* slots;  // read when not fused
  const int32_t* bt;
  const int32_t* offs;
  const int32_t* tok_seq;
  const int32_t* tok_pos;
  int64_t* slots_out;  // fused: also written here when not null
  int mb, batch;
};

// Slot of token t from its (sequence, position): -1 for padding (negative
// sequence) and for anything out of range (recorded in the error word when
// `report`).
__device__ __forceinline__ int64_t token_slot(const SlotSrc& ss, long long t, long long num_blocks,
                                              int bs, int* err, bool report) {
  const int b = ss.tok_seq[t];
  if (b < 0) return -1;
  if (b >= ss.batch) {
    if (report) set_error(err, kErrIndex);
    return -1;
  }
  const int off = ss.offs ? ss.offs[b] : 0;
  const long long p = (long long)off + ss.tok_pos[t];
  if (off < 0 || off >= bs || ss.tok_pos[t] < 0 || p >= (long long)ss.mb * bs) {
    if (report) set_error(err, kErrCapacity);
    return -1;
  }
  // block sizes are powers of two: a shift instead of a 64-bit division
  const int shift = 31 - __clz(bs);
  const int blk = ss.bt[(long long)b * ss.mb + (p >> shift)];
  if (blk < 0 || blk >= num_blocks) {
    if (report) set_error(err, kErrIndex);
    return -1;
  }
  return ((int64_t)blk << shift) + (p & (bs - 1));
}

}  // namespace pkv
