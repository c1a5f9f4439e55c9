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

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}
__device__ __forceinline__ int wave_scan(int v, int lane) {   // inclusive
  for (int o = 1; o < kWave; o <<= 1) {
    const int u = __shfl_up(v, o, kWave);
    if (lane >= o) v += u;
  }
  return v;
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

}  // namespace nvfp4moe
