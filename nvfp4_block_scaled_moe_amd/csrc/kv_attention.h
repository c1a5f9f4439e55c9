// Pieces shared by the kernels of the attention over the paged cache: which rows and keys a
// workgroup takes, what a row sees, conversions and lane moves.
#pragma once

#include "common.h"
#include "kernels.h"
#include "kv_division.h"

namespace nvfp4moe {

typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f;

// First key that the row of a position sees (no sum here passes 32 bits, whatever the window).
__device__ __forceinline__ int first_seen(int position, int window) {
  return window > 0 && position >= window ? position - window + 1 : 0;
}

// One sequence's new tokens.
struct Sequence {
  int row0, n;       // first row, new tokens (rows within the tensor only)
  int len;           // tokens, the new ones among them
  int cap;           // keys that the page table has columns for
  int blocks;        // of the keys that any of them sees
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
  const int last = min(q.len, q.cap), first = first_seen(q.len - q.n, window);
  q.blocks = max(blocks_of(last, block_log) - (first >> block_log), 0);
  return q;
}

// Keys a row sees: those in [lo, hi).
struct Seen {
  int lo, hi;
};
__device__ __forceinline__ Seen seen_by(int position, int window, int cap) {
  return {first_seen(position, window), min(max(position + 1, 0), cap)};
}

// What the sums of new token i's row are multiplied by, `total` being that of its weights: zeros where it sees no key, which
// is where it lies before its sequence; NaN where the page table has no column for it. A row that sees keys has a
// total above 0 unless all its scores are -Inf: 0 / 0, NaN, as its softmax.
__device__ __forceinline__ float normalize(const Sequence& q, int i, float total, float v_scale) {
  const int p = q.position(i);
  return p < 0 ? 0.0f : p >= q.cap ? NAN : v_scale / total;
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

struct Segment {
  Sequence seq;
  int s, tile;            // the sequence, its row tile
  int parts, part;        // of the tile's keys
  int slot;               // place of this part's sums, where parts > 1 (heads aside)
  int block0, blocks;     // this part's keys
  bool found;
};
// Segment `at` (heads aside), or with SPLIT tile `at` of those that are split (part 0). (Rows of a sequence are below
// 2^27 and blocks below 2^27: every division is of 32 bits.)
template <bool SPLIT>
__device__ __forceinline__ Segment segment_of(const KvAttnArgs& p, const Division& v, int at) {
  const CacheBatchArgs& b = p.batch;
  const int lane = threadIdx.x % kWave;   // a lane a sequence
  auto tiles_of = [&](const Sequence& q) { return (q.n * p.G + v.tile_rows() - 1) >> v.tile_log; };
  Sequence mine{};
  int64_t work = 0;
  for (int s0 = 0; s0 < b.B; s0 += kWave) {
    const int s = s0 + lane;
    if (s < b.B) {
      mine = sequence_of(b, p.window, s, v.block_log);
      work += (int64_t)tiles_of(mine) * mine.blocks;
    }
  }
  work = wave_sum(work) * p.Hkv;
  const int64_t even = (work + (1 << v.target_log) - 1) >> v.target_log;
  const uint32_t chunk = (uint32_t)min((even > v.min_blocks ? even : v.min_blocks), (int64_t)1 << 30);
  Segment r{};
  int before = 0, slots = 0;
  for (int s0 = 0; s0 < b.B; s0 += kWave) {
    const int s = s0 + lane;
    if (b.B > kWave) mine = s < b.B ? sequence_of(b, p.window, s, v.block_log) : Sequence{};
    const int tiles = s < b.B ? tiles_of(mine) : 0, parts = parts_of((uint32_t)mine.blocks, chunk);
    const int split = parts > 1 ? tiles * parts : 0, count = SPLIT ? (parts > 1 ? tiles : 0) : tiles * parts;
    const int upto = wave_scan(count), split_upto = wave_scan(split);
    const uint64_t hit = __ballot(before + upto > at);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      auto get = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
      r.seq = {get(mine.row0), get(mine.n), get(mine.len), get(mine.cap), get(mine.blocks)};
      r.s = s0 + l;
      r.parts = get(parts);
      const int in = at - before - (get(upto) - get(count)), nth = SPLIT ? in : in / r.parts;
      r.part = SPLIT ? 0 : in - nth * r.parts;
      r.tile = get(tiles) - 1 - nth;   // (the later ones, which see the most, first)
      r.slot = slots + get(split_upto) - get(split) + nth * r.parts + r.part;
      // the blocks that the tile's rows see
      const int t0 = (int)((uint32_t)(r.tile << v.tile_log) / (uint32_t)p.G);
      const int t1 = min((int)((uint32_t)((r.tile << v.tile_log) + v.tile_rows() - 1) / (uint32_t)p.G), r.seq.n - 1);
      const Seen a = seen_by(r.seq.position(t0), p.window, r.seq.cap), z = seen_by(r.seq.position(t1), p.window, r.seq.cap);
      r.block0 = a.lo >> v.block_log;
      r.blocks = max(blocks_of(z.hi, v.block_log) - r.block0, 0);
      if (!SPLIT) {
        const int per = ((r.blocks + r.parts - 1) / r.parts + v.step - 1) / v.step * v.step;
        r.block0 += r.part * per;
        r.blocks = max(min(per, r.blocks - r.part * per), 0);   // (the last parts may have none)
      }
      r.found = true;
      return r;
    }
    before += __builtin_amdgcn_readlane(upto, kWave - 1);
    slots += __builtin_amdgcn_readlane(split_upto, kWave - 1);
  }
  return r;
}

// Sums of a part in the workspace: [slot, head] of [tile_rows, D] unnormalised outputs, then of
// [tile_rows] maxima (of base 2 logits) and sums.
struct Sums {
  float* o;
  float* ml;
  __device__ __forceinline__ Sums(const KvAttnArgs& p, const Division& v, int64_t slot, int h) {
    const int64_t i = slot * p.Hkv + h;
    o = static_cast<float*>(p.ws) + i * v.tile_rows() * (p.D + 2);
    ml = o + v.tile_rows() * p.D;
  }
};

// Joins the parts of a tile: a workgroup takes `turns` times `together` of its rows for one head, of which each
// thread holds 4 dims of every groups-th part; in a fixed order. Where little is split, what this costs is finding
// that out in every workgroup (8192 of them 13 us, 2048 6 to 8), so there are no more than the CUs hold at once.
constexpr int kJoinThreads = 256, kJoinGroups = 2048;
namespace {   // (a kernel of each file's own)
template <bool FP8, class Of>   // Of::kDivision
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const KvAttnArgs p, int together, int turns) {
  constexpr Division v = Of::kDivision;
  __shared__ float4 s_o[kJoinThreads];
  __shared__ float2 s_ml[kJoinThreads];
  const int sets = v.tile_rows() / (together * turns), h = blockIdx.x / sets % p.Hkv;
  const Segment sg = segment_of<true>(p, v, blockIdx.x / sets / p.Hkv);
  if (!sg.found) return;
  const int lanes = p.D / 4, groups = kJoinThreads / (lanes * together);
  const int lane = threadIdx.x % lanes, group = threadIdx.x / lanes % groups;
  const int rows = sg.seq.n * p.G - (sg.tile << v.tile_log);   // of the tile and those behind it
  for (int turn = 0; turn < turns; ++turn) {
    const int r0 = (blockIdx.x % sets * turns + turn) * together, r = r0 + threadIdx.x / (lanes * groups);
    if (r0 >= rows) return;
    const bool mine = (int)threadIdx.x < lanes * groups * together && r < rows;
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float2 ml, float4 x) {
      const float next = fmaxf(m, ml.x), base = next == -INFINITY ? 0.0f : next;
      const float f = __builtin_amdgcn_exp2f(m - base), e = ml.x == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(ml.x - base);
      m = next;
      l = l * f + ml.y * e;
      o.x = o.x * f + x.x * e, o.y = o.y * f + x.y * e, o.z = o.z * f + x.z * e, o.w = o.w * f + x.w * e;
    };
    if (mine)
#pragma unroll 4
      for (int i = group; i < sg.parts; i += groups) {
        const Sums part(p, v, sg.slot + i, h);
        add(*reinterpret_cast<const float2*>(part.ml + 2 * r), *reinterpret_cast<const float4*>(part.o + r * p.D + 4 * lane));
      }
    if (groups > 1) {
      if (turn > 0) __syncthreads();   // what the turn before left is read
      s_o[threadIdx.x] = o;
      s_ml[threadIdx.x] = make_float2(m, l);
      __syncthreads();
    }
    if (!mine || group > 0) continue;
    for (int i = 1; i < groups; ++i) add(s_ml[threadIdx.x + i * lanes], s_o[threadIdx.x + i * lanes]);
    const int at = (sg.tile << v.tile_log) + r, t = at / p.G;
    const float f = normalize(sg.seq, t, l, FP8 && p.v_scale ? p.v_scale[h] : 1.0f);
    uint16_t* to = p.out + (sg.seq.row0 + t) * p.o_row + (h * p.G + at - t * p.G) * p.o_head + 4 * lane;
    *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2(o.x * f, o.y * f), bf16x2(o.z * f, o.w * f));
  }
}
template <bool FP8, class Of>
hipError_t launch_join(const KvAttnArgs& a, hipStream_t stream) {
  constexpr Division v = Of::kDivision;
  if (!v.can_split((int64_t)a.batch.cols << a.batch.page_log)) return hipSuccess;
  const int64_t tiles = v.split_tiles(a.batch.T, a.batch.B, a.Hkv, a.G);
  // rows that a workgroup joins at once: one, or as many as its threads hold where that leaves a few workgroups a CU
  int together = 1, turns = 1;
  while (together * 2 * (a.D / 4) <= kJoinThreads && tiles * a.Hkv * (v.tile_rows() / (2 * together)) >= 1024) together *= 2;
  while (together * turns < v.tile_rows() && tiles * a.Hkv * (v.tile_rows() / (together * turns)) > kJoinGroups) turns *= 2;
  const int64_t sets = tiles * a.Hkv * (v.tile_rows() / (together * turns));
  join_kernel<FP8, Of><<<dim3((unsigned)sets), kJoinThreads, 0, stream>>>(a, together, turns);
  return hipGetLastError();
}
}  // namespace

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

// Eight E4M3 bytes as f16 (exact).
__device__ __forceinline__ f16x8 e4m3x8_to_f16(uint32_t a, uint32_t b) {
  const f16x2 p = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false), q = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
  const f16x2 r = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false), s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
  return (f16x8){p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
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
  const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // bit 7 of each that is NaN
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
