// How the work of the attention over the paged cache is divided between workgroups: the arithmetic that the host, which
// launches, and the kernels, which find their shares by it, have in common. Nothing here is the device's alone, so
// that a host compiler can check what each may take for granted of the other.
#pragma once

#include <cstddef>
#include <cstdint>

#ifdef __HIPCC__
#define NVFP4MOE_BOTH __host__ __device__
#else
#define NVFP4MOE_BOTH
#endif

namespace nvfp4moe {

// Blocks that hold `keys` keys, and parts that a tile of `blocks` is split into (1: it is not).
template <class Int>
NVFP4MOE_BOTH constexpr Int blocks_of(Int keys, int block_log) {
  return (keys + (1 << block_log) - 1) >> block_log;
}
NVFP4MOE_BOTH constexpr int parts_of(uint32_t blocks, uint32_t chunk) {
  const uint32_t n = (blocks + chunk / 2) / chunk;
  return n > 1 ? (int)n : 1;
}

// How the work is divided. Rows (token, head of a group) of a sequence and key head are taken in tiles, their
// keys in blocks; the tiles of a sequence are split into as many parts each as its blocks are whole segments,
// rounded, a segment being the target's share of all blocks of all tiles (counted as if every tile saw what its
// sequence sees), or min_blocks. Every wave finds its segment by itself from the lengths: they are known
// on the device alone, and a launch that lists the segments costs more (6 to 9 us).
struct Division {
  int tile_log, block_log;
  int target_log;   // segments that the work is divided into
  int min_blocks;   // least blocks of one
  int step;         // parts are multiples of it
  // A sequence is split from 1.5 segments on, so at most 2 / 3 of the target's tiles are split, into at
  // most 4 / 3 of its segments; all segments are at most the tiles and the target.
  NVFP4MOE_BOTH constexpr int tile_rows() const { return 1 << tile_log; }
  NVFP4MOE_BOTH constexpr int split_blocks() const { return min_blocks + min_blocks / 2; }
  // Whether a sequence can be split whose page table holds `keys` tokens: its blocks, which bound those of any length
  // and window, and shares of min_blocks, which are the least.
  NVFP4MOE_BOTH constexpr bool can_split(int64_t keys) const { return blocks_of(keys, block_log) >= split_blocks(); }
  int64_t tiles(int T, int B, int G) const { return ((int64_t)T * G + tile_rows() - 1) / tile_rows() + (B < T ? B : T); }
  int64_t whole(int Hkv) const { return ((int64_t(1) << target_log) + Hkv - 1) / Hkv; }   // of the target, heads aside
  int64_t segments(int T, int B, int Hkv, int G) const { return tiles(T, B, G) + whole(Hkv); }
  int64_t split_tiles(int T, int B, int Hkv, int G) const {
    const int64_t n = tiles(T, B, G), w = whole(Hkv);
    return n < w ? n : w;
  }
  size_t ws_bytes(int Hkv, int D) const { return (size_t)(4 * whole(Hkv) / 3 + 1) * Hkv * tile_rows() * (D + 2) * sizeof(float); }
};

// Of tiles of 16 rows (kv_attention_few.hip), whose waves take every fourth block. (Least blocks of a segment: joining
// costs a second launch, so that a few blocks more a wave cost less.)
constexpr int kFewWaves = 4;
constexpr Division few_division(bool fp8) { return {4, fp8 ? 6 : 5, 10, 16, kFewWaves}; }

// Of tiles of 128 and 256 rows (kv_attention.hip), W waves to a workgroup: 4, two workgroups a CU, or 8, one a CU, whose
// tiles bring half the words for a row. The segments are as many as workgroups that the CUs hold at once. With W 4, 512
// and 1024 of them: 16 sequences of 4 tokens over 8000 keys 103 and 111 us, E4M3 66 and 74; two E4M3 sequences of 1 and
// 4 tokens over 90000 to 130000 109 and 117; 2048 tokens over 6000 of D 256 668 and 716; whole prompts, windows and D 64
// the same. (640 and 768, which leave a part round: 125 and 115 us for the first, which took 105 then.)
constexpr int kChunkBlockLog = 6;   // keys of a block
constexpr Division chunk_division(int W) { return {W == 8 ? 8 : 7, kChunkBlockLog, W == 8 ? 8 : 9, 8, 1}; }

}  // namespace nvfp4moe
