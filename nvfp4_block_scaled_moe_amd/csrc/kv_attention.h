// Pieces shared by the kernels of the attention over the paged cache: which rows and keys a
// workgroup takes, what a row sees, conversions and lane moves.
#pragma once

#include "common.h"
#include "kernels.h"

namespace nvfp4moe {

typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f;

// One sequence's new tokens, and the blocks of keys that any of them sees.
struct Sequence {
  int row0, n;       // first row, new tokens (rows within the tensor only)
  int len;           // tokens, the new ones among them
  int cap;           // keys that the page table has columns for
  int block0, blocks;
  // Position of new token i, and the first key that it sees.
  __device__ __forceinline__ int position(int i) const { return len - n + i; }
};
// block_log: keys of a block. A sequence longer than its page table gives NaN in the rows that
// would see keys behind it; nothing behind it is read.
__device__ __forceinline__ Sequence sequence_of(const CacheBatchArgs& b, int window, int s, int block_log) {
  Sequence q;
  const int start = b.starts[s], end = b.starts[s + 1], len = b.lengths[s];
  q.row0 = min(max(start, 0), b.T);
  q.n = max(min(end, b.T) - q.row0, 0);
  q.len = max(len, 0);
  q.cap = (int)min((int64_t)b.cols << b.page_log, (int64_t)0x7fffff00);
  const int last = min(q.len, q.cap), first = window > 0 ? max(q.len - q.n + 1 - window, 0) : 0;
  q.block0 = first >> block_log;
  q.blocks = max(((last + (1 << block_log) - 1) >> block_log) - q.block0, 0);
  return q;
}

// Keys a row sees: those in [lo, hi).
struct Seen {
  int lo, hi;
};
__device__ __forceinline__ Seen seen_by(int position, int window, int cap) {
  return {window > 0 ? max(position + 1 - window, 0) : 0, min(max(position + 1, 0), cap)};
}

// Inclusive sums over the lanes by DPP moves (no LDS round trips): within rows of 16, then rows 1 and 3
// take the row before, then rows 2 and 3 the first half's.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);    // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast31
  return v;
}
// Sum over the lanes of values in [0, 2^55), the same in all.
__device__ __forceinline__ int64_t wave_sum(int64_t v) {
  const int lo = __builtin_amdgcn_readlane(wave_scan((int)(v & 0xffffff)), kWave - 1);
  const int hi = __builtin_amdgcn_readlane(wave_scan((int)(v >> 24)), kWave - 1);
  return ((int64_t)hi << 24) + lo;
}

// Four E4M3 bytes as bf16 (exact).
__device__ __forceinline__ u32x2 e4m3x4_to_bf16(uint32_t w) {
  const bf16x2v lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
  const bf16x2v hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true);
  return {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}
__device__ __forceinline__ bf16x8 e4m3x8_to_bf16(uint32_t a, uint32_t b) {
  const u32x2 x = e4m3x4_to_bf16(a), y = e4m3x4_to_bf16(b);
  return __builtin_bit_cast(bf16x8, (u32x4v){x[0], x[1], y[0], y[1]});
}

// For values that only some of a tile's rows see: a product with a zero weight must not let a NaN or
// Inf into the rows that do not see it. Two bf16 (a word) with those replaced by 0; `bad` gets a bit
// pattern that is not zero for each of them.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w, uint32_t& bad) {
  const uint32_t lo = (w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u, hi = (w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
  bad = lo | hi;
  return w & ~bad;
}

// Four E4M3 bytes with NaN (0x7f, 0xff) replaced by 0.
__device__ __forceinline__ uint32_t finite_e4m3x4(uint32_t w) {
  uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // bit 7 of each that is NaN
  return w & ~(nan | (nan - (nan >> 7)));
}

// max of a lane's value and those of the lanes 16, 32 and 48 on
__device__ __forceinline__ float max_of_groups(float v) {
  const u32x2 a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const u32x2 b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

}  // namespace nvfp4moe
