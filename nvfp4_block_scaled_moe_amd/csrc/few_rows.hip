// Products of a few rows with FP4 weights (gfx950): the matrix-vector products nvfp4_matvec and
// mxfp4_matvec, and the whole mixture-of-experts layer of up to 16 tokens in two launches
// (moe_layer_few_nvfp4, moe_layer_few_mxfp4).
//
//   matvec      out[t, n] = sum_k x[t, k] W[n, k] (* g) (+ add), or silu(gate) * up (+ add)
//   layer, 1st  route the T tokens, h[r, f] = silu(x_t Wg_e^T)[f] * (x_t Wu_e^T)[f] for the row
//               r of every kept (token t, expert e)
//   layer, 2nd  out[t, n] = sum over t's experts of w(t, e) * sum_f h[r, f] W2_e[n, f]
//
// Every weight byte is used by at most 16 rows, so the bound is the HBM rate on codes and
// scales (9/16 or 17/32 byte a weight), and for small matrices the latency of a chain of dependent
// steps. The kernels read each weight once and keep two or three of each wave's loads under way:
//
//   * A wave streams 16-row x 128-column tiles (1 KB of codes in the order of the matrix
//     core's operand, weights_tile.hip) into a ring of registers, with the lane's scale bytes
//     beside them. One workgroup of 16 waves a CU: what a CU can have under way is limited, so all
//     256 have to take the same number of bytes, and its older waves are served first, so the
//     waves meet at a barrier once a tile (or a turn of the ring).
//   * The columns of a tile are dealt out to the waves chunk by chunk, so that a single 16-row
//     tile keeps a CU busy; the waves' float32 sums meet in LDS once a tile, in a fixed order.
//   * Persistent workgroups walk a contiguous range of tiles as one flat sequence of chunks: the
//     ring stays full across tiles and experts.
//   * NVFP4 weights are decoded exactly to f16 (E2M1 * E4M3 has at most 6 significant bits), so the
//     rows become f16, scaled by a power of two so that a row's (or, where the row does not fit in
//     LDS, its chunk's) largest finite magnitude lies in [2^14, 2^15): exact for bf16 values down
//     to 2^-31 of that magnitude; the sums take the power back. MXFP4 weights are decoded exactly to
//     bf16 (whose exponent holds every E8M0 scale), so bf16 rows are used as they are.
//   * The layer's first launch routes in every workgroup (a wave per token; a few microseconds
//     that replace a launch), the second reads the list that one of them left. An item is an
//     expert with up to 4 of its tokens; an expert with more tokens takes several items.
//   * h between the launches: f16 with a power of two for each 16 columns (NVFP4: 11 bits of what
//     is then summed in float32), or two bf16 values, the second what the first's rounding left
//     (MXFP4: 16 bits; their matrix operand is bf16, and with its 8 bits alone the layer's error is
//     0.0024 instead of the 0.0017 of its bf16 output. The second values' products cost 2-5%: 16
//     tokens of 256 experts 353 -> 360 us, one 40.6 -> 41.4, 2 of 60 21.3 -> 22.1).
//   * The second launch adds a token's experts in its accumulators, in a fixed order: no
//     float32 rows of the experts go through memory, and no reduce launch follows.
#include <hip/hip_runtime.h>

#include "act_rows.h"
#include "gemm_common.h"
#include "kernels.h"
#include "route_token.h"

namespace nvfp4moe {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kW = 16;                   // waves per workgroup: a CU's worth at 128 registers
constexpr int kNT = kW * kWave;
constexpr int kGrid = 256;               // persistent workgroups: one on each of the 256 CUs
constexpr int kLongW = 8;                // waves per workgroup of few_long_kernel
constexpr int kLongNT = kLongW * kWave;
constexpr int kRowBytes = 256 + 16;      // LDS bytes of one row's chunk (padded: conflict-free reads)
constexpr int kDownLeast = 128;          // pairs of the second launch that are worth a workgroup: sharing a
                                         // tile costs 2-4 us (layers of one token of 256 experts, 128 pairs a
                                         // tile, 45.8 us, shared from 24, 48 or 80 pairs on 47.7-47.9; of 2
                                         // tokens of 60, 2080 x 1376, 21.3 us, shared 24.9-25.9)
constexpr int kItemTok = 4;              // tokens of one item of the layer
template <bool B>
struct Flag {
  static constexpr bool value = B;
};
constexpr int kNoExp = -120;             // exponent of a block of h without a finite non-zero value

// ------------------------------------------------------------------ operand decode
// Eight E2M1 codes times an E8M0 scale (as a float: 2^(s-127), NaN for 0xFF) as bf16, exact.
__device__ __forceinline__ bf16x8 decode8_mx(uint32_t w, float s) {
  const bf16x2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  const bf16x2v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  const bf16x2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  const bf16x2v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return (bf16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ float e8m0_to_f32(uint32_t s) {
  const uint32_t bits = s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23;
  return __uint_as_float(bits);
}

__host__ __device__ __forceinline__ int nch_of(int K) { return (K + kChunk - 1) / kChunk; }

// Max over the 16 lanes of a row, in all of them.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
#pragma unroll
  for (int s = 0; s < 4; ++s) v = dpp_max_u32(v, s);
  return v;
}

// The matrix operands of one weight tile (16 rows x 128 columns): codes w, the lane's scale bytes.
template <bool MX>
struct Decode;
template <>
struct Decode<false> {
  typedef f16x8 Op;
  static __device__ __forceinline__ void run(const u32x4& w, uint32_t sv, Op (&o)[4]) {
    f16x2 s0, s1;
    decode_scale_pair(sv, s0, s1);
    o[0] = decode8(w[0], s0);
    o[1] = decode8(w[1], s0);
    o[2] = decode8(w[2], s1);
    o[3] = decode8(w[3], s1);
  }
  // One quarter of it (dword j of the lane's codes).
  static __device__ __forceinline__ Op part(uint32_t w, uint32_t sv, int j) {
    const f16 s = (f16)e4m3_to_f32(j < 2 ? sv & 0xffu : (sv >> 8) & 0xffu);
    return decode8(w, (f16x2){s, s});
  }
  static __device__ __forceinline__ f32x4 mfma(const Op& a, const Op& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Decode<true> {
  typedef bf16x8 Op;
  static __device__ __forceinline__ void run(const u32x4& w, uint32_t sv, Op (&o)[4]) {
    const float s = e8m0_to_f32(sv);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = decode8_mx(w[j], s);
  }
  static __device__ __forceinline__ Op part(uint32_t w, uint32_t sv, int) { return decode8_mx(w, e8m0_to_f32(sv)); }
  static __device__ __forceinline__ f32x4 mfma(const Op& a, const Op& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

// Offset of the dword that holds the lane's scale bytes of (16-row block blk, chunk c) in the
// tiled scales, and the bytes taken out of it. (Whole dwords: a narrower load's zero extension
// would be placed, and waited for, at the end of the loop body instead of at its use.)
template <bool MX>
__device__ __forceinline__ uint32_t scale_off(uint32_t c) {   // in a row block's tiles
  return MX ? (c >> 4) * 1024u + (c & 12) : (c >> 3) * 1024u + 2u * (c & 6);
}
template <bool MX>
__device__ __forceinline__ uint32_t scale_off(uint32_t blk, uint32_t nch, uint32_t c) {
  return blk * (MX ? (nch + 15) >> 4 : (nch + 7) >> 3) * 1024u + scale_off<MX>(c);
}
template <bool MX>
__device__ __forceinline__ uint32_t scale_of(uint32_t dword, uint32_t c) {
  return MX ? (dword >> (8u * (c & 3))) & 0xffu : dword >> (16u * (c & 1));
}
__device__ __forceinline__ uint32_t ld32(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff = 0) {
  return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
}
// An offset as a value of its own: keeps the compiler from turning a select of offsets into
// branches with a load in each, after which it could only wait for all loads at once.
__device__ __forceinline__ uint32_t settled(uint32_t off) {
  asm("" : "+v"(off));
  return off;
}
__device__ __forceinline__ int settled_s(int v) {   // (the same in every lane)
  v = __builtin_amdgcn_readfirstlane(v);
  asm("" : "+s"(v));
  return v;
}

// A matrix's global scale g = rest * power, power = 2^n, 1 <= |rest| < 2 (a normal g). Sums over
// chunks that have powers of two of their own take `power` with each chunk, so that what they hold
// is within a factor 2 of the result: without g it would be some 2^15 times that, and rows near
// 2^118 whose result is finite would overflow. `least` is the smallest exponent of a chunk whose
// power times 2^n is exact (2^-149, float32's smallest value): a chunk below it is scaled by less,
// and what its f16 loses lies below float32's smallest values in the result, too.
struct GlobalScale {
  float power, rest;
  uint32_t least;
  __device__ __forceinline__ explicit GlobalScale(float g) {
    const uint32_t e = min(__float_as_uint(g) >> 23 & 0xffu, 254u);   // n + 127
    power = __uint_as_float(e ? e << 23 : 0x00400000u);
    rest = ldexpf(g, 127 - (int)e);
    least = (uint32_t)max(15, 119 - (int)e);
  }
};

// Eight bf16 elements of each of two rows' chunks, a chunk held by 16 lanes together, as f16
// scaled by a power of two of the chunk; unscale is the power that takes it back, times that of the
// global scale. (Two rows a call: the steps of one fill the waits of the other's reduction.)
__device__ __forceinline__ void chunks_to_f16(const u32x4& v0, const u32x4& v1, const GlobalScale& gs, f16x8 (&o)[2],
                                              float (&unscale)[2]) {
  uint32_t top[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const u32x4& v = r ? v1 : v0;
    u16x2 m = __builtin_bit_cast(u16x2, v[0] & 0x7fff7fffu);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu));
    top[r] = max((uint32_t)m[0], (uint32_t)m[1]);
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    top[0] = dpp_max_u32(top[0], s);
    top[1] = dpp_max_u32(top[1], s);
  }
  if (__ballot(max(top[0], top[1]) >= 0x7f80u)) {   // an Inf or NaN somewhere: the maximum over the finite ones
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const u32x4& v = r ? v1 : v0;
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = v[i] & 0x7fffu, hi = (v[i] >> 16) & 0x7fffu;
        t = max(t, lo < 0x7f80u ? lo : 0u);
        t = max(t, hi < 0x7f80u ? hi : 0u);
      }
      top[r] = row16_max(t);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const u32x4& v = r ? v1 : v0;
    const uint32_t eb = max(top[r] >> 7, gs.least);   // biased exponent of the maximum
    const float scale = __uint_as_float((268u - eb) << 23);
    unscale[r] = __uint_as_float((eb - 14u) << 23) * gs.power;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[r][2 * i] = (f16)(bf16_to_f32(v[i] & 0xffffu) * scale);
      o[r][2 * i + 1] = (f16)(__uint_as_float(v[i] & 0xffff0000u) * scale);
    }
  }
}

// A chunk of up to 16 rows, row 4 r + (lane >> 4) in x[r], as matrix operands to `row` (LDS, 16 rows
// of kRowBytes) and its powers of two to `unscale`; x loaded as zeros past the T rows.
template <bool MX>
__device__ __forceinline__ void put_rows(const u32x4 (&x)[4], int T, int lane, const GlobalScale& gs, unsigned char* row,
                                         float* unscale) {
  const int l16 = lane & 15, g = lane >> 4;
#pragma unroll
  for (int r = 0; r < 4; r += 2) {
    if (4 * r >= T) continue;
    unsigned char* at = row + (4 * r + g) * kRowBytes + 16 * l16;
    if (MX) {
      *reinterpret_cast<u32x4*>(at) = x[r];
      *reinterpret_cast<u32x4*>(at + 4 * kRowBytes) = x[r + 1];
    } else {
      f16x8 o[2];
      float un[2];
      chunks_to_f16(x[r], x[r + 1], gs, o, un);
      *reinterpret_cast<f16x8*>(at) = o[0];
      *reinterpret_cast<f16x8*>(at + 4 * kRowBytes) = o[1];
      if (l16 == 0) {
        unscale[4 * r + g] = un[0];
        unscale[4 * r + 4 + g] = un[1];
      }
    }
  }
}

// Power of two (as a float) that takes a row's largest finite magnitude, given as bf16 bits,
// into [2^14, 2^15), and the one that takes it back.
__device__ __forceinline__ uint32_t row_exponent(uint32_t top) { return max(top >> 7, 15u); }
__device__ __forceinline__ float row_scale(uint32_t top) { return __uint_as_float((268u - row_exponent(top)) << 23); }
__device__ __forceinline__ float row_unscale(uint32_t top) { return __uint_as_float((row_exponent(top) - 14u) << 23); }
// Largest magnitude below `end` of eight bf16 values, as bf16 bits (0x7f80: of the finite ones,
// 0x7f81: Inf counts).
__device__ __forceinline__ uint32_t top_of(const u32x4& v, uint32_t end) {
  u16x2 m = __builtin_bit_cast(u16x2, v[0] & 0x7fff7fffu);
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu));
  uint32_t t = max((uint32_t)m[0], (uint32_t)m[1]);
  if (__ballot(t >= end)) {   // some are not to be counted
    t = 0;
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = i < 4 ? (i < 2 ? v[0] : v[1]) : (i < 6 ? v[2] : v[3]);
      const uint32_t a = (i & 1 ? w >> 16 : w) & 0x7fffu;
      t = max(t, a < end ? a : 0u);
    }
  }
  return t;
}
__device__ __forceinline__ f16x8 scaled_f16(const u32x4& v, float scale) {
  f16x8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = (f16)(bf16_to_f32(v[i] & 0xffffu) * scale);
    o[2 * i + 1] = (f16)(__uint_as_float(v[i] & 0xffff0000u) * scale);
  }
  return o;
}

// fp8_roundtrip_bits of two bf16 values (packed low, high), as packed bf16: the quotient v / s
// as (float)((double)v * inv) with inv the double nearest 1 / s. That rounds correctly: the
// product is within 2^-52 of v / s, and v / s, with v of 8 and s of 24 significant bits, is never
// within 2^-49 of the middle of two floats. Infinite values go to the largest code; NaN stays.
__device__ __forceinline__ uint32_t fp8_pair(uint32_t w, float s, double inv) {
  float q[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float v = __uint_as_float(i ? w & 0xffff0000u : w << 16);
    const float r = (float)((double)v * inv);
    q[i] = v != v ? v : fminf(fmaxf(r, -448.0f), 448.0f);
  }
  const f32x2 f = __builtin_amdgcn_cvt_pk_f32_fp8(__builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false), false);
  return bf16x2(f[0] * s, f[1] * s);
}

// First column block of wave group rg's b-th row block in a tile: gate blocks, then their up blocks.
template <bool SWIGLU, int RB>
__device__ __forceinline__ uint32_t tile_block(uint32_t sub, int b, uint32_t nblk) {
  return SWIGLU ? sub * (RB / 2) + b % (RB / 2) + (b < RB / 2 ? 0 : nblk / 2) : sub * RB + b;
}
// Whether that block exists: the last tile may be short.
template <bool SWIGLU, int RB>
__device__ __forceinline__ bool tile_block_in(uint32_t sub, int b, uint32_t nblk) {
  return SWIGLU ? sub * (RB / 2) + b % (RB / 2) < nblk / 2 : sub * RB + b < nblk;
}

// The output of one element of a matvec.
__device__ __forceinline__ void put_matvec(const FewArgs& p, int col, size_t n0, float v) {
  if (p.add) {
    const size_t ao = (size_t)col * p.ld_add + n0;
    v += p.add_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.add)[ao]) : static_cast<const float*>(p.add)[ao];
  }
  const size_t o = (size_t)col * p.ld_out + n0;
  if (p.out_bf16)
    static_cast<__bf16*>(p.out)[o] = (__bf16)v;
  else
    static_cast<float*>(p.out)[o] = v;
}

// What every wave does once before its first load is paid sixteen times over: the four waves of a
// SIMD share one scalar unit and take turns (four cycles an instruction), and the code comes from a
// cold instruction cache (about 2 bytes a nanosecond). So: 32 bits, no division by a variable (25
// instructions each).
//
// x / d from inv = floor(2^32 / d), at most 2^32 - 1 (inverse() below): x inv / 2^32 is less than
// x / d by at most x / 2^32 < 1, so that its whole part is the quotient or one less.
__device__ __forceinline__ uint32_t quotient(uint32_t x, uint32_t d, uint32_t inv) {
  const uint32_t q = (uint32_t)(((uint64_t)x * inv) >> 32);
  return q + (x - q * d >= d ? 1u : 0u);
}

// An even split of `total` things over n takers, the first `more` of them with one more.
struct Share {
  uint32_t each, more;
  __device__ __forceinline__ Share(uint32_t total, uint32_t n, uint32_t each_) : each(each_), more(total - each_ * n) {}
  __device__ __forceinline__ Share(uint32_t each_, uint32_t more_) : each(each_), more(more_) {}
  __device__ __forceinline__ uint32_t begin(uint32_t i) const { return i * each + (i < more ? i : more); }
  // The taker of thing x.
  __device__ __forceinline__ uint32_t taker(uint32_t x) const {
    const uint32_t edge = more * (each + 1);
    return x < edge ? x / (each + 1) : more + (x - edge) / each;
  }
};

// Inclusive sum over the lanes before, by lane moves: within rows of 16, then the rows' totals.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false);   // row_bcast 15, 31
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false);
  return v;
}

// The kernel's arguments, one of each 64 bytes of them, requested together: the first reading of
// each misses every cache (a microsecond), and the compiler would leave some to where they are used.
__device__ __forceinline__ void fetch_args(const FewArgs& p) {
  static_assert(sizeof(FewArgs) <= 192, "three lines");
  asm volatile("" ::"s"(p.K), "s"(p.grid), "s"(p.most_parts));
}

// ------------------------------------------------------------------ resident rows: matvec, and the layer's first launch
// The rows (the item's, or all of them once when they fit) stay in LDS as matrix operands, f16
// with one power of two a row (NVFP4) or bf16 (MXFP4): turned once, they serve every tile of
// the item. Waves deal out the chunks ks at a time (ks = 1 .. 16: kW / ks groups of
// waves, each with RB row blocks of its own).
//
// Measured (the kernel alone, weights cold). Products: 2048 x 6144, one row, 7.1 MB: 6.8 us;
// 2064 x 1184, MXFP4, 5 rows, 1.3 MB: 4.9 us; SwiGLU 1024 x 256, one row: 4.7 us. These are
// latency: ~1 us of launch and arguments, 2 us until the rows are operands, 2 us until the weights
// are there, 1 us of sums and stores; a CU alone draws about 45 B/ns. The layer: 16 tokens of 256
// experts, 6144 x 2048, 1.43 GB: 245-251 us, 5.8 TB/s, where plain reads reach 6.0-6.5; one token of it,
// 113 MB: 26 us, of which 4-5 are routing and staging and 2 the last tile's sums; 3 tokens of 8, 256 x
// 512: 7.3 us.
// 16-byte pieces of the rows a thread requests together: one row seldom has more than one for each.
constexpr int pass_batch(int ntok) { return ntok > 4 ? 4 : 1; }

template <bool MX, bool LAYER, bool FP8, bool SWIGLU, int NTOK, int D>
__global__ __launch_bounds__(kNT, 4) void few_up_kernel(const FewArgs p) {
  typedef Decode<MX> Dec;
  typedef typename Dec::Op Op;
  constexpr int RB = SWIGLU ? 2 : 1;   // row blocks of a wave: one, or a gate block and its up block
  static_assert(!LAYER || (SWIGLU && NTOK == kItemTok), "the layer's items");
  static_assert(!FP8 || (LAYER && !MX), "FP8 activations: the NVFP4 layer");
  constexpr int BUF = NTOK > 4 ? 1 : 2;
  constexpr int kPassBatch = pass_batch(NTOK);
  constexpr int REDF = kW * RB * NTOK * 16;
  extern __shared__ __attribute__((aligned(16))) unsigned char s_rows[];   // [rows][K128 * 2 + 16]
  __shared__ __attribute__((aligned(16))) float s_red[BUF][REDF];
  __shared__ uint32_t s_top[NTOK];                          // largest finite magnitude of each row
  __shared__ uint32_t s_item[LAYER ? kFewMaxSlots : 1];     // expert << 16 | token mask
  __shared__ uint16_t s_row0[LAYER ? kFewMaxSlots : 1];     // first row of the item in h
  __shared__ uint32_t s_first[LAYER ? kMaxExperts : 1];     // token mask, then item << 16 | row
  __shared__ int s_ids[LAYER ? kFewMaxSlots : 1];
  __shared__ float s_w[LAYER ? kFewMaxSlots : 1];
  __shared__ uint32_t s_scan[kW];
  __shared__ uint32_t s_amax;

  fetch_args(p);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int T = p.T, K = p.K;
  const uint32_t nch = (uint32_t)(K + kChunk - 1) / kChunk;
  const uint32_t stride = nch * 256u + 16u;              // LDS bytes of a row
  static_assert(kW == 16, "4 - ks_log");
  const int KS = 1 << p.ks_log, rg_log = 4 - p.ks_log, RG = 1 << rg_log;
  const int ksl = wave & (KS - 1), rg = wave >> p.ks_log;
  const int cpw = ((int)nch + KS - 1) >> p.ks_log;       // chunks of a tile for each wave
  const uint32_t nblk = (uint32_t)p.Nw / 16;             // row blocks of a matrix
  const int nsub = (int)nblk / RB;                       // groups: a row block, or a gate block and its up block
  const int tpi = (nsub + RG - 1) >> rg_log;             // tiles of an item
  const uint32_t wbytes = nblk * nch * 1024u;
  const uint32_t sbytes = nblk * (MX ? (nch + 15) >> 4 : (nch + 7) >> 3) * 1024u;
  const bool all_rows = !LAYER || T <= p.item_tok;       // every row fits: staged once

  // ---- rows (all_rows: every row, else those of mask) into LDS, by nt threads (this one the
  // first-th), in batches of kPassBatch pieces a thread: their largest magnitudes (find_tops),
  // then, after a barrier, the operands (put_rows). A second reading, from the caches, is needed
  // only for rows of more than one batch.
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x, (uint32_t)((p.ldx * (T - 1) + K) * 2));
  const uint32_t ppr = nch * 16u;   // 16-byte pieces of a row
  auto row_at = [&](uint32_t piece) { return __umulhi(piece, p.ppr_inv); };   // piece / ppr (host: ppr_inverse)
  u32x4 pv[kPassBatch];
  auto load_batch = [&](uint32_t mask, uint32_t total, uint32_t i0, uint32_t nt) {
#pragma unroll
    for (int i = 0; i < kPassBatch; ++i) {
      const uint32_t idx = i0 + i * nt, r = row_at(idx), q = idx - r * ppr;
      uint32_t tok = r;
      if (LAYER && !all_rows) {
        uint32_t m = mask;
#pragma unroll
        for (uint32_t j = 0; j < (uint32_t)kItemTok - 1; ++j) m = j < r ? m & (m - 1) : m;
        tok = (uint32_t)__ffs(m) - 1u;
      }
      const bool in = idx < total && 8u * q < (uint32_t)K;
      pv[i] = ld128(xr, settled(in ? tok * (uint32_t)p.ldx * 2u + 16u * q : kOOB), 0);
    }
  };
  uint32_t amax = 0;   // FP8: the largest finite magnitude that this thread has seen
  auto tops_of_batch = [&](uint32_t total, uint32_t i0, uint32_t nt) {
#pragma unroll
    for (int i = 0; i < kPassBatch; ++i) {
      const uint32_t idx = i0 + i * nt;
      const uint32_t top = row16_max(top_of(pv[i], FP8 ? 0x7f81u : 0x7f80u));   // (a row's pieces come in sixteens)
      if (l16 == 0 && idx < total) atomicMax(&s_top[row_at(idx)], top);
      if (FP8) amax = max(amax, top_of(pv[i], 0x7f80u));
    }
  };
  auto find_tops = [&](uint32_t mask, uint32_t total, uint32_t first, uint32_t nt) {
    for (uint32_t i0 = first; i0 < total; i0 += kPassBatch * nt) {
      load_batch(mask, total, i0, nt);
      tops_of_batch(total, i0, nt);
    }
  };
  float fp8_s = 1.0f;
  double fp8_inv = 1.0;
  // FP8: the first n rows' largest magnitudes as they are after the round trip (which keeps the order).
  auto fp8_tops = [&](int n) {
    if (FP8) {
      if (tid < n) s_top[tid] = fp8_pair(s_top[tid], fp8_s, fp8_inv) & 0x7fffu;
      __syncthreads();
    }
  };
  auto put_batch = [&](uint32_t total, uint32_t i0, uint32_t nt) {
#pragma unroll
    for (int i = 0; i < kPassBatch; ++i) {
      const uint32_t idx = i0 + i * nt, r = row_at(idx);
      if (idx < total) {
        unsigned char* at = s_rows + r * stride + 16u * (idx - r * ppr);
        if (MX) {
          *reinterpret_cast<u32x4*>(at) = pv[i];
        } else {
          u32x4 v = pv[i];
          if (FP8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = fp8_pair(v[j], fp8_s, fp8_inv);
          }
          *reinterpret_cast<f16x8*>(at) = scaled_f16(v, row_scale(s_top[r]));
        }
      }
    }
  };
  auto put_rows = [&](uint32_t mask, uint32_t total, uint32_t first, uint32_t nt) {
    if (total <= kPassBatch * nt) {   // find_tops (MXFP4: load_batch) has left them in registers
      put_batch(total, first, nt);
    } else {
      for (uint32_t i0 = first; i0 < total; i0 += kPassBatch * nt) {
        load_batch(mask, total, i0, nt);
        put_batch(total, i0, nt);
      }
      // Every load has arrived: without the wait here the compiler would place it in the main
      // loop, for the lanes that used none of theirs.
      __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    }
  };

  int nitems = 1;
  const uint32_t all = all_rows ? (uint32_t)T * ppr : 0u;   // pieces staged once
  // The threads that stage them: in the layer those of the waves that route no token (all of
  // them when every wave does).
  const uint32_t st0 = LAYER && T < kW ? (uint32_t)T * kWave : 0u;
  const uint32_t stn = (uint32_t)kNT - st0;
  if (tid < NTOK) s_top[tid] = 0;
  if constexpr (LAYER) {
    // ---- routing: a wave per token
    static_assert(BUF * REDF >= kW * 3 * kWave, "the routing scratch fits");
    static_assert(kFewMaxTokens <= kW, "a wave per token");
    const int E = p.E, k = p.k, S = T * k;
    if (S > kWave)
      for (int e = tid; e < E; e += kNT) s_first[e] = 0;
    if (FP8 && tid == 0) s_amax = 0;
    __syncthreads();
    if (wave < T) {
      const float* row = p.logits + (size_t)wave * E;
      uint32_t* scratch = reinterpret_cast<uint32_t*>(&s_red[0][0]) + wave * 3 * kWave;
      auto route = [&](auto regs) {   // (top-16 and up without serial rounds, as the router does)
        constexpr int PL = decltype(regs)::value;
        if (k < 16)
          route_token_rounds<PL, false>(row, E, k, lane, s_ids + wave * k, s_w + wave * k, nullptr);
        else
          route_token_thresh<PL, false>(row, E, k, lane, s_ids + wave * k, s_w + wave * k, nullptr, scratch);
      };
      if (E <= kWave)
        route(Int<1>{});
      else if (E <= 256)
        route(Int<4>{});
      else if (E <= 512)
        route(Int<8>{});
      else
        route(Int<16>{});
      if (T == 1 && lane < k) {   // an item for each kept expert (the wave's own LDS accesses keep their order)
        s_item[lane] = (uint32_t)s_ids[lane] << 16 | 1u;
        s_row0[lane] = (uint16_t)lane;
      }
    }
    if (MX && all && (uint32_t)tid >= st0) load_batch(0, all, (uint32_t)tid - st0, stn);
    if (!MX && (uint32_t)tid >= st0) {
      if (all) find_tops(0, all, (uint32_t)tid - st0, stn);
      if (FP8 && !all_rows) {   // the scale is taken over every row
        const uint32_t total = (uint32_t)T * ppr;
        for (uint32_t i = (uint32_t)tid - st0; i < total; i += stn) {
          const uint32_t t = row_at(i), q = i - t * ppr;
          const u32x4 v = ld128(xr, settled(8u * q < (uint32_t)K ? t * (uint32_t)p.ldx * 2u + 16u * q : kOOB), 0);
          amax = max(amax, top_of(v, 0x7f80u));
        }
      }
      if (FP8) {
        amax = row16_max(amax);
        if (l16 == 0) atomicMax(&s_amax, amax);
      }
    }
    __syncthreads();
    if (FP8) {
      fp8_s = fp8_scale(bf16_to_f32(s_amax));
      fp8_inv = 1.0 / (double)fp8_s;
      if (all_rows) fp8_tops(T);
    }
    const uint32_t cap = (uint32_t)p.item_tok;
    if (T == 1) {
      nitems = k;
    } else if (S <= kWave) {
      // ---- the items in ascending expert order, by one wave with a lane for each slot (slots of
      // an expert ascend with their tokens): for each slot the lanes with its expert, and with
      // smaller ones; every cap-th slot of an expert starts an item
      if (wave == 0) {
        const uint32_t k_inv = 65536u / (uint32_t)k + 1u;   // (slots below 64: exact)
        const int e = lane < S ? s_ids[lane] : 0x7fffffff;
        uint32_t same[2] = {0, 0}, less[2] = {0, 0};
        for (int j = 0; j < S; ++j) {
          const int ej = __builtin_amdgcn_readlane(e, j);
          const uint64_t eq = __ballot(e == ej), lt = __ballot(e < ej);
          const bool mine = lane == j;
          same[0] = mine ? (uint32_t)eq : same[0];
          same[1] = mine ? (uint32_t)(eq >> 32) : same[1];
          less[0] = mine ? (uint32_t)lt : less[0];
          less[1] = mine ? (uint32_t)(lt >> 32) : less[1];
        }
        const uint64_t eq = (uint64_t)same[1] << 32 | same[0], lt = (uint64_t)less[1] << 32 | less[0];
        const uint32_t before = (uint32_t)__popcll(eq & ((1ull << lane) - 1ull));
        const uint32_t part = before * (cap == 1 ? 12u : cap == 2 ? 6u : cap == 3 ? 4u : 3u) / 12u;   // before / cap
        const bool starts = lane < S && part * cap == before;
        const uint64_t first = __ballot(starts);
        if (starts) {
          const uint32_t item = (uint32_t)__popcll(lt & first) + part, row = (uint32_t)__popcll(lt) + before;
          uint64_t rest = eq >> lane << lane;   // the expert's slots from this one on
          uint32_t tokens = 0;
          for (uint32_t j = 0; j < cap && rest; ++j) {
            tokens |= 1u << ((uint32_t)__builtin_ctzll(rest) * k_inv >> 16);
            rest &= rest - 1;
          }
          s_item[item] = (uint32_t)e << 16 | tokens;
          s_row0[item] = (uint16_t)row;
          if (part == 0) s_first[e] = item << 16 | row;
        }
        if (lane == 0) s_scan[0] = (uint32_t)__popcll(first);
      }
      __syncthreads();
      nitems = (int)s_scan[0];
    } else {
      // ---- the items in ascending expert order
      for (int s = tid; s < S; s += kNT) atomicOr(&s_first[s_ids[s]], 1u << (s / k));
      __syncthreads();
      // a thread for each expert: the items and rows before its own by a scan over the threads
      static_assert(kMaxExperts <= kNT, "a thread for each expert");
      uint32_t m = tid < E ? s_first[tid] : 0u;
      const uint32_t rows = (uint32_t)__popc(m);
      // (ceil(rows / cap) for cap 1 .. 4 and at most 16 rows)
      const uint32_t cnt = ((rows + cap - 1) * (cap == 1 ? 12u : cap == 2 ? 6u : cap == 3 ? 4u : 3u) / 12u) << 16 | rows;
      const uint32_t incl = wave_scan(cnt);
      if (lane == kWave - 1) s_scan[wave] = incl;
      __syncthreads();
      uint32_t at = incl - cnt, sum = 0;
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const uint32_t v = s_scan[w];
        at += w < wave ? v : 0u;
        sum += v;
      }
      nitems = (int)(sum >> 16);
      if (m) {
        s_first[tid] = at;
        while (m) {
          uint32_t rest = m;   // m without its lowest `cap` tokens
          for (uint32_t j = 0; j < cap; ++j) rest &= rest - 1;
          const uint32_t part = m & ~rest;
          s_item[at >> 16] = (uint32_t)tid << 16 | part;
          s_row0[at >> 16] = (uint16_t)(at & 0xffffu);
          at += 0x10000u + (uint32_t)__popc(part);
          m = rest;
        }
      }
      __syncthreads();
    }
    nitems = __builtin_amdgcn_readfirstlane(nitems);
  }

  auto write_plan = [&]() {   // the list for the second launch
    const int k = p.k;
    if (wave < T) {   // the kept experts' softmax, of the logits that the routing left (largest first)
      const float x = lane < k ? s_w[wave * k + lane] : 0.0f;
      const float top = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 0));
      const float ex = lane < k ? expf(x - top) : 0.0f;
      float sum = ex;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
      if (lane < k) s_w[wave * k + lane] = ex / sum;
    }
    __syncthreads();
    for (int i = tid; i < nitems; i += kNT) p.plan->item[i] = s_item[i];
    for (int i = tid; i < nitems; i += kNT) p.plan->row0[i] = s_row0[i];
    if (tid == 0) p.plan->n_items = nitems;
    for (int i = tid; i < p.down_tiles; i += kNT) p.plan->arrived[i] = 0;
    for (int s = tid; s < T * k; s += kNT) {
      const int t = s / k, e = s_ids[s];
      int at = s;   // T == 1: the rows in the kept order
      if (T > 1) {
        const uint32_t before = (1u << t) - 1u;   // tokens before t with the same expert
        at = (int)(s_first[e] & 0xffffu);
        for (int i = (int)(s_first[e] >> 16); i < nitems && (int)(s_item[i] >> 16) == e; ++i)
          at += __popc(s_item[i] & before);
      }
      p.plan->weight[at] = MX ? s_w[s] : s_w[s] * p.g_down[e];
    }
  };

  // ---- this workgroup's tiles, in runs of one item's: a flat sequence of steps (a chunk of RB
  // weight tiles), D of them a turn of the ring. A tile takes at least D steps, so that at most
  // one is completed in a turn; a run is padded to whole turns.
  const uint32_t ntile = (uint32_t)nitems * (uint32_t)tpi;
  const Share share(ntile, (uint32_t)p.grid, quotient(ntile, (uint32_t)p.grid, p.grid_inv));
  const int t0 = (int)share.begin(blockIdx.x), t1 = (int)share.begin(blockIdx.x + 1);
  if (t0 >= t1) return;   // fewer tiles than workgroups

  __amdgpu_buffer_rsrc_t wr, sr;
  auto item_word = [&](int it) -> uint32_t {
    return LAYER ? (uint32_t)__builtin_amdgcn_readfirstlane((int)s_item[it]) : (1u << T) - 1u;
  };
  const uint32_t wrow = nch * 1024u, srow = (MX ? (nch + 15) >> 4 : (nch + 7) >> 3) * 1024u;   // of a row block
  const uint32_t half = nblk / 2;   // SwiGLU: from a group's gate block to its up block
  // The chunk of a wave runs from ksl in steps of KS; a tile takes cpw of them, or D.
  const uint32_t cend = (uint32_t)ksl + ((uint32_t)(cpw > D ? cpw : D) << p.ks_log);
  const int spt = cpw > D ? cpw : D;   // steps of a tile
  // Of a run of n tiles from `tile` on, those in which this wave has a group of row blocks (the
  // last tile's groups may end before it).
  auto tiles_of = [&](int tile, int n) { return min(n, (nsub - tile * RG - rg + RG - 1) >> rg_log); };
  // The loads' position: the item and the tiles left behind the run; in the run the tile, of n_l,
  // and its first block's bytes; and the chunk.
  int it_l = LAYER ? (int)quotient((uint32_t)t0, (uint32_t)tpi, p.tpi_inv) : 0;
  int tile_l = t0 - it_l * tpi, tiles_l = t1 - t0, at_l = 0, n_l = 0, own_l = 0;
  uint32_t c_l = 0, woff_l = 0, soff_l = 0;
  const uint32_t wstep = (uint32_t)RG * wrow, sstep = (uint32_t)RG * srow;
  auto open_run = [&]() {
    const size_t e = LAYER ? item_word(it_l) >> 16 : 0;
    wr = make_rsrc(p.codes + e * wbytes, wbytes);
    sr = make_rsrc(p.scales + e * sbytes, sbytes);
    n_l = min(tiles_l, tpi - tile_l);
    tiles_l -= n_l;
    at_l = 0;
    own_l = tiles_of(tile_l, n_l);
    c_l = (uint32_t)ksl;
    woff_l = (uint32_t)(tile_l * RG + rg) * wrow;
    soff_l = (uint32_t)(tile_l * RG + rg) * srow;
    tile_l = 0;
    ++it_l;
  };
  u32x4 wring[D][RB];
  uint32_t sring[D][RB];
  const uint32_t lane16 = 16u * lane;
  auto issue = [&](int d) {
    // A step without a chunk loads from out of range. (Its scalar offset is 0: one past the
    // resource's end would wrap the hardware's comparison.) All in sign masks: of selects the
    // compiler makes branches, a load in each, or sends the position through memory.
    const int in = settled_s((int)(c_l - nch) & (at_l - own_l));   // negative: there is a chunk
    const uint32_t v = settled(lane16 | (kOOB & ~(uint32_t)in)), all = (uint32_t)(in >> 31);
    const uint32_t w0 = (woff_l + c_l * 1024u) & all, s0 = (soff_l + scale_off<MX>(c_l)) & all;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      wring[d][b] = ld128(wr, v, w0 + (b ? half * wrow & all : 0u));
      sring[d][b] = ld32(sr, v, s0 + (b ? half * srow & all : 0u));
    }
    c_l += (uint32_t)KS;
    const uint32_t wrap = ~(uint32_t)settled_s((int)(c_l - cend) >> 31);   // all ones at the tile's end
    c_l -= wrap & (cend - (uint32_t)ksl);
    at_l -= (int)wrap;
    woff_l += wrap & wstep;
    soff_l += wrap & sstep;
  };

  int it = it_l, tile = tile_l, left = t1 - t0, buf = 0, done = 0;
  open_run();
  // Fill the ring. (After each turn the next run is opened where this one's loads have ended.)
  auto next_run = [&]() {
    if (at_l >= n_l && tiles_l > 0) open_run();
  };
  // The layer's rows have arrived and go to LDS first (a wave whose loads find no room waits for
  // the others' to return); a matvec's are requested first and looked at behind the ring's loads.
  if (LAYER && all) {
    if ((uint32_t)tid >= st0) put_rows(0, all, (uint32_t)tid - st0, stn);
    __syncthreads();
  }
  if (!LAYER) load_batch(0, all, (uint32_t)tid, stn);
#pragma unroll
  for (int d = 0; d < D; ++d) issue(d);
  next_run();
  if (!LAYER) {
    if (!MX) {
      __syncthreads();   // s_top is cleared
      tops_of_batch(all, (uint32_t)tid, stn);
      if (all > kPassBatch * stn) find_tops(0, all, (uint32_t)tid + kPassBatch * stn, stn);
      __syncthreads();
    }
    put_rows(0, all, (uint32_t)tid, stn);
    __syncthreads();
  }
  if constexpr (LAYER) {
    if (blockIdx.x == 0) write_plan();   // (the first workgroup always has a tile)
  }

  f32x4 tot[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) tot[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
  for (bool first = true; left > 0; first = false) {
    const uint32_t word = item_word(it);
    const int ncol = __popc(word & 0xffffu);
    if (LAYER && !all_rows) {
      const uint32_t m = word & 0xffffu, total = (uint32_t)ncol * ppr;
      if (!first) {
        __syncthreads();   // the last epilogue has read the last item's rows
        if (tid < NTOK) s_top[tid] = 0;
        __syncthreads();
      }
      if (MX) {
        load_batch(m, total, (uint32_t)tid, kNT);
      } else {
        find_tops(m, total, (uint32_t)tid, kNT);
        __syncthreads();
        fp8_tops(ncol);
      }
      put_rows(m, total, (uint32_t)tid, kNT);
      __syncthreads();
    }
    // The staged row of column col (the col-th token of the item; the last one past them).
    auto row_of = [&](int col) -> uint32_t {
      const int q = col < ncol ? col : ncol - 1;
      if (!LAYER || !all_rows) return (uint32_t)q;
      uint32_t rest = word & 0xffffu;
      for (int j = 0; j < q; ++j) rest &= rest - 1;
      return (uint32_t)__builtin_ctz(rest);
    };
    const uint32_t frow = settled(row_of(l16) * stride + 64u * g);
    const float alpha = MX ? 1.0f : ld_const(p.g, LAYER ? word >> 16 : 0);
    const int run = min(left, tpi - tile), own = tiles_of(tile, run);
    left -= run;
    int at = 0;
    uint32_t c = (uint32_t)ksl;
    for (int steps = run * spt; steps > 0; steps -= D) {
      int ready = 0;
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (c < nch && at < own) {
          Op bf[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) bf[j] = *reinterpret_cast<const Op*>(s_rows + frow + c * 256u + 16 * j);
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            Op wf[4];
            Dec::run(wring[d][b], scale_of<MX>(sring[d][b], c), wf);
#pragma unroll
            for (int j = 0; j < 4; ++j) tot[b] = Dec::mfma(wf[j], bf[j], tot[b]);
          }
        }
        issue(d);
        c += (uint32_t)KS;
        const bool wrap = c == cend;
        c = wrap ? (uint32_t)ksl : c;
        if (wrap && at++ < run) {   // a tile is complete: this wave's sums
          ready = 1;
          if (l16 < NTOK) {
#pragma unroll
            for (int b = 0; b < RB; ++b)
              *reinterpret_cast<f32x4*>(&s_red[buf][((wave * RB + b) * NTOK + l16) * 16 + 4 * g]) = tot[b];
          }
#pragma unroll
          for (int b = 0; b < RB; ++b) tot[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
        }
      }
      next_run();
      if (ready) {
        // ---- the waves' sums together, and the epilogue
        __syncthreads();
        const float* red = s_red[buf];
        const int lcol = ncol > 1 ? 32 - __builtin_clz(ncol - 1) : 0;   // columns, to a power of two
        const int total = (RG * 16) << lcol;
        // a different wave starts each tile, so that short epilogues spread over the SIMDs
        for (int i = (tid + kWave * done) & (kNT - 1); i < total; i += kNT) {
          const int r16 = i & 15, q = i >> 4;
          const int grp = q >> lcol, col = q & ((1 << lcol) - 1);
          if (col >= ncol) continue;   // (16 lanes at a time)
          const int osub = tile * RG + grp;
          float v = 0.0f, u = 0.0f;
          // (the waves' values are requested four at a time; what is past KS is not added)
          for (int w0 = 0; w0 < KS; w0 += 4) {
            float av[4], au[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float* a = &red[(((grp * KS + (w0 + w < KS ? w0 + w : w0)) * RB) * NTOK + col) * 16 + r16];
              av[w] = a[0];
              au[w] = SWIGLU ? a[NTOK * 16] : 0.0f;
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              v += w0 + w < KS ? av[w] : 0.0f;
              if (SWIGLU) u += w0 + w < KS ? au[w] : 0.0f;
            }
          }
          const float un = MX ? 1.0f : row_unscale(s_top[row_of(col)]);
          v = v * alpha * un;
          if (SWIGLU) v = swiglu1(v, u * alpha * un);
          if constexpr (LAYER) {
            const uint32_t hr = (uint32_t)s_row0[it] + (uint32_t)col;
            const int F = p.Nw / 2, f = osub * 16 + r16;
            if (MX) {
              if (osub < nsub) {   // (rows [2][F]: the value, and what its rounding left)
                const __bf16 hi = (__bf16)v;
                __bf16* at = static_cast<__bf16*>(p.h) + (size_t)hr * 2 * F + f;
                at[0] = hi;
                at[F] = fabsf((float)hi) < INFINITY ? (__bf16)(v - (float)hi) : (__bf16)0.0f;
              }
            } else {
              const uint32_t top = row16_max(finite_abs_bits(v));
              const int e2 = top ? max((int)(top >> 23) - 141, kNoExp) : kNoExp;
              if (osub < nsub) {
                static_cast<f16*>(p.h)[(size_t)hr * F + f] = (f16)ldexpf(v, -e2);
                if (r16 == 0) p.hexp[(size_t)hr * (nch_of(F) * 8) + osub] = (int8_t)e2;
              }
            }
          } else if (osub < nsub) {
            put_matvec(p, col, (size_t)osub * 16 + r16, v);
          }
        }
        if (BUF == 1) __syncthreads();
        else buf ^= 1;
        ++done;
        ++tile;
      }
    }
    tile = 0;
    ++it;
  }
}

// ------------------------------------------------------------------ matvec of rows that do not fit
// Up to 16 rows of any length: the 8 waves of a workgroup (two a CU) deal out the chunks and each
// turns its chunk of the rows itself, in a piece of LDS of its own, with a power of two for every
// (row, chunk). The turning costs about as much as the decode of four weight tiles, and is most of
// the time where there are few weight rows: 2048 x 6144 with 16 rows 9.6 us, MXFP4 7.3 (not turned).
// Far from the reads' bound at ordinary sizes, 6144 columns: 8192 weight rows 12.2 us (of 5.6), MXFP4
// 9-11 (5.3), 16384 20.9 (11.2) and 17-18 (10.6): the rows are turned again for each tile, and with
// two row blocks a wave one chunk is under way.
template <bool MX, bool SWIGLU, int RB, int D>
__global__ __launch_bounds__(kLongNT, 4) void few_long_kernel(const FewArgs p) {
  typedef Decode<MX> Dec;
  typedef typename Dec::Op Op;
  constexpr int R = kFewMaxTokens / 4;
  constexpr int HB = SWIGLU ? RB / 2 : RB;
  __shared__ __attribute__((aligned(16))) unsigned char s_row[kLongW][kFewMaxTokens * kRowBytes];
  __shared__ float s_unscale[kLongW][kFewMaxTokens];
  __shared__ __attribute__((aligned(16))) float s_red[kLongW * RB][16 * 16];

  fetch_args(p);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int T = p.T, K = p.K;
  const uint32_t nch = (uint32_t)nch_of(K);
  const int cpw = ((int)nch + kLongW - 1) / kLongW;
  const uint32_t nblk = (uint32_t)p.Nw / 16;
  const int ntiles = ((int)(SWIGLU ? nblk / 2 : nblk) + HB - 1) / HB;
  const uint32_t wbytes = nblk * nch * 1024u;
  const uint32_t sbytes = nblk * (MX ? (nch + 15) >> 4 : (nch + 7) >> 3) * 1024u;
  const int t0 = (int)((int64_t)ntiles * blockIdx.x / p.grid);
  const int t1 = (int)((int64_t)ntiles * (blockIdx.x + 1) / p.grid);
  const int nst = (t1 - t0) * cpw;

  const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x, (uint32_t)((p.ldx * (T - 1) + K) * 2));
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(p.codes, wbytes), sr = make_rsrc(p.scales, sbytes);
  uint32_t xoff[R];
#pragma unroll
  for (int r = 0; r < R; ++r) xoff[r] = 4 * r + g < T ? (uint32_t)((4 * r + g) * p.ldx * 2) + 16u * l16 : kOOB;

  u32x4 wring[D][RB], xring[D][R];
  uint32_t sring[D][RB];
  int tile_l = t0, step_l = 0, left_l = nst;   // the loads' position
  // A tile's blocks are refilled one by one as they are consumed, the rows' pieces before them.
  uint32_t c_l = 0;
  bool ok_l = false;
  auto issue_rows = [&](int d) {
    c_l = (uint32_t)(wave + step_l * kLongW);
    ok_l = left_l > 0 && c_l < nch;
    const bool cols = ok_l && (int)(c_l * kChunk) + 8 * l16 < K;
#pragma unroll
    for (int r = 0; r < R; ++r) xring[d][r] = ld128(xr, settled(cols ? xoff[r] + c_l * 256u : kOOB), 0);
  };
  auto issue_block = [&](int d, int b) {
    const uint32_t blk = tile_block<SWIGLU, RB>(tile_l, b, nblk);
    const bool in = ok_l && tile_block_in<SWIGLU, RB>(tile_l, b, nblk);
    wring[d][b] = ld128(wr, settled(16u * lane + (in ? (blk * nch + c_l) * 1024u : kOOB)), 0);
    sring[d][b] = ld32(sr, settled(16u * lane + (in ? scale_off<MX>(blk, nch, c_l) : kOOB)));
  };
  auto issue_end = [&]() {
    --left_l;
    const int wrap = step_l + 1 == cpw ? 1 : 0;
    step_l = wrap ? 0 : step_l + 1;
    tile_l += wrap;
  };
#pragma unroll
  for (int d = 0; d < D; ++d) {
    issue_rows(d);
#pragma unroll
    for (int b = 0; b < RB; ++b) issue_block(d, b);
    issue_end();
  }

  const GlobalScale gs(MX ? 1.0f : ld_const(p.g, 0));
  f32x4 tot[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) tot[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
  unsigned char* row = s_row[wave];
  int tile = t0, step = 0;
  for (int s = 0; s < nst; s += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      // (chunks past the last have loaded zeros, rows and weights, and add nothing)
      const uint32_t c = (uint32_t)(wave + step * kLongW);
      put_rows<MX>(xring[d], T, lane, gs, row, s_unscale[wave]);
      issue_rows(d);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      Op bf[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) bf[j] = *reinterpret_cast<const Op*>(row + l16 * kRowBytes + 64 * g + 16 * j);
      const float un = MX ? 1.0f : s_unscale[wave][l16];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        Op wf[4];
        Dec::run(wring[d][b], scale_of<MX>(sring[d][b], c), wf);
        issue_block(d, b);
        f32x4 a = MX ? tot[b] : (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) a = Dec::mfma(wf[j], bf[j], a);
        if (MX) {
          tot[b] = a;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[b][i] = fmaf(a[i], un, tot[b][i]);
        }
      }
      issue_end();
      step += s + d < nst ? 1 : 0;
      if (step == cpw) {
        step = 0;
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          *reinterpret_cast<f32x4*>(&s_red[wave * RB + b][l16 * 16 + 4 * g]) = tot[b];
          tot[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
        }
        __syncthreads();
        for (int i = tid; i < HB * T * 16; i += kLongNT) {
          const int r16 = i & 15, q = i >> 4, b = q / T, col = q - b * T;
          if (!tile_block_in<SWIGLU, RB>(tile, b, nblk)) continue;
          float v = 0.0f, u = 0.0f;
#pragma unroll
          for (int w = 0; w < kLongW; ++w) {
            v += s_red[w * RB + b][col * 16 + r16];
            if (SWIGLU) u += s_red[w * RB + b + HB][col * 16 + r16];
          }
          v *= gs.rest;
          if (SWIGLU) v = swiglu1(v, u * gs.rest);
          put_matvec(p, col, (size_t)tile_block<SWIGLU, RB>(tile, b, nblk) * 16 + r16, v);
        }
        __syncthreads();
        ++tile;
      }
    }
  }
}

// Rows that do not fit, many weight rows: a wave owns RB row blocks over all of K, so that no sums
// cross waves, and the W waves of a workgroup share the rows: each of them turns one of the next W
// chunks into operands, in the other half of a double-buffered piece of LDS.
//
// Between two bounds: the vector units are busy half the time (79 instructions a tile and wave, 32
// of them the decoding, 25 the rows), and the reads go at three quarters of the memory's rate. 65536 x
// 6144 at 16 rows: 47.7 us, 4.8 TB/s (MXFP4 43); few_long_kernel, in which every wave turns its own
// chunks, 71; 16 waves sharing (half the turning, but all of a CU's waves at one barrier) 50; two
// row blocks a wave 51; two or eight chunks under way 52 and 50.
template <bool MX, bool SWIGLU, int RB, int W, int D>
__global__ __launch_bounds__(W* kWave, 4) void few_wide_kernel(const FewArgs p) {
  typedef Decode<MX> Dec;
  typedef typename Dec::Op Op;
  static_assert(!SWIGLU || RB == 2, "a gate block and its up block");
  static_assert(W % D == 0, "ring entries return to the same place in every group");
  constexpr int R = kFewMaxTokens / 4;
  __shared__ __attribute__((aligned(16))) unsigned char s_row[2][W][kFewMaxTokens * kRowBytes];
  __shared__ float s_unscale[2][W][kFewMaxTokens];

  fetch_args(p);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int T = p.T, K = p.K;
  const uint32_t nch = (uint32_t)nch_of(K);
  const int ngroups = ((int)nch + W - 1) / W;
  const uint32_t nblk = (uint32_t)p.Nw / 16;
  const uint32_t wrow = nch * 1024u, srow = (MX ? (nch + 15) >> 4 : (nch + 7) >> 3) * 1024u;   // of a row block
  const uint32_t sub = blockIdx.x * W + wave;                                                   // this wave's blocks
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x, (uint32_t)((p.ldx * (T - 1) + K) * 2));
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(p.codes, nblk * wrow), sr = make_rsrc(p.scales, nblk * srow);
  uint32_t xoff[R];
#pragma unroll
  for (int r = 0; r < R; ++r) xoff[r] = 4 * r + g < T ? (uint32_t)((4 * r + g) * p.ldx * 2) + 16u * l16 : kOOB;

  u32x4 wring[D][RB], xv[R];
  uint32_t sring[D][RB];
  auto issue_rows = [&](uint32_t c) {
    const bool cols = c * kChunk + 8 * l16 < (uint32_t)K;
#pragma unroll
    for (int r = 0; r < R; ++r) xv[r] = ld128(xr, settled(cols ? xoff[r] + c * 256u : kOOB), 0);
  };
  auto issue = [&](int d, uint32_t c) {
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const uint32_t blk = tile_block<SWIGLU, RB>(sub, b, nblk);
      const bool in = c < nch && tile_block_in<SWIGLU, RB>(sub, b, nblk);
      wring[d][b] = ld128(wr, settled(16u * lane + (in ? blk * wrow + c * 1024u : kOOB)), 0);
      sring[d][b] = ld32(sr, settled(16u * lane + (in ? blk * srow + scale_off<MX>(c) : kOOB)));
    }
  };
  const GlobalScale gs(MX ? 1.0f : ld_const(p.g, 0));
  auto put_chunk = [&](int buf) { put_rows<MX>(xv, T, lane, gs, s_row[buf][wave], s_unscale[buf][wave]); };
  issue_rows((uint32_t)wave);
#pragma unroll
  for (int d = 0; d < D; ++d) issue(d, (uint32_t)d);
  f32x4 tot[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) tot[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
  put_chunk(0);
  __syncthreads();
  for (int gr = 0; gr < ngroups; ++gr) {
    const int buf = gr & 1;
    // (chunks past the last have loaded zeros, rows and weights, and add nothing)
    issue_rows((uint32_t)((gr + 1) * W + wave));
#pragma unroll 1
    for (int u0 = 0; u0 < W; u0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int u = u0 + d;
        const uint32_t c = (uint32_t)(gr * W + u);
        const float un = MX ? 1.0f : s_unscale[buf][u][l16];
        f32x4 a[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) a[b] = MX ? tot[b] : (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const Op bf = *reinterpret_cast<const Op*>(s_row[buf][u] + l16 * kRowBytes + 64 * g + 16 * j);
#pragma unroll
          for (int b = 0; b < RB; ++b)
            a[b] = Dec::mfma(Dec::part(wring[d][b][j], scale_of<MX>(sring[d][b], c), j), bf, a[b]);
          if (RB == 2 && j == 1) __builtin_amdgcn_sched_barrier(0);   // (all four operands at once would spill)
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          if (MX) {
            tot[b] = a[b];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[b][i] = fmaf(a[b][i], un, tot[b][i]);
          }
        }
        issue(d, c + D);
        __builtin_amdgcn_sched_barrier(0);   // (the next chunk's reads moved up here would cost the ring its registers)
      }
    }
    put_chunk(buf ^ 1);
    __syncthreads();
  }
  if (l16 < T) {
    constexpr int NB = SWIGLU ? 1 : RB;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (!tile_block_in<SWIGLU, RB>(sub, b, nblk)) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = tot[b][i] * gs.rest;
        if (SWIGLU) v = swiglu1(v, tot[RB - 1][i] * gs.rest);
        put_matvec(p, l16, (size_t)tile_block<SWIGLU, RB>(sub, b, nblk) * 16 + 4 * g + i, v);
      }
    }
  }
}

// ------------------------------------------------------------------ the layer's second launch
// A tile is RB row blocks, 16 or 32 output columns; its work is the (item, chunk) pairs. The
// pairs of all tiles form one sequence that the workgroups share evenly (whole tiles seldom give
// every CU the same number of bytes: 192 tiles on 256 CUs, three quarters of the rate), unless the
// parts would be short (kDownLeast). A tile that several workgroups have part of is finished by the
// last of them to arrive, which adds the parts in order; nobody waits.
//
// A wave's pair needs up to four rows' chunk of h beside the weights, brought to the row's common
// exponent on its way through LDS. Measured: 16 tokens of 256 experts, 6144 x 2048, 0.71 GB:
// 136 us, 5.2 TB/s; one token, 57 MB: 17.0 us, of which 3 pass until the list is read and the
// ring is full and 2-3 in the last sums; 2 tokens of 60, 2080 x 1376, MXFP4, 12 MB: 9.3 us; 3 of 8,
// 256 x 512: 5.3 us. Keeping the ring full over a tile's end (the next tile's loads under its sums)
// brought nothing when the layer of one token took 50.4 us: 50.9.
template <bool MX, int RB>
__global__ __launch_bounds__(kNT, 4) void few_down_kernel(const FewArgs p) {
  constexpr int D = 2;   // chunks of a wave under way (3: a per cent or two slower, 4: spills)
  typedef Decode<MX> Dec;
  typedef typename Dec::Op Op;
  static_assert(kFewMaxSlots <= kNT, "a thread for each row and item");
  __shared__ __attribute__((aligned(16))) unsigned char s_row[kW][(MX ? 2 : 1) * kItemTok * kRowBytes];
  __shared__ __attribute__((aligned(16))) float s_red[kW * RB][16 * 16];
  __shared__ uint32_t s_item[kFewMaxSlots];
  __shared__ uint16_t s_row0[kFewMaxSlots];
  __shared__ float s_mul[kFewMaxSlots];   // what a row's products are multiplied with
  __shared__ int s_top[kFewMaxSlots];     // NVFP4: the largest exponent of a row's blocks
  __shared__ int s_last;

  fetch_args(p);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int T = p.T, F = p.K, S = T * p.k;
  const uint32_t nch = (uint32_t)nch_of(F);
  const uint32_t nblk = (uint32_t)p.Nw / 16;
  const uint32_t wbytes = nblk * nch * 1024u;
  const uint32_t sbytes = nblk * (MX ? (nch + 15) >> 4 : (nch + 7) >> 3) * 1024u;

  // The list of items (its first entries are read beside their number), and what each row is
  // multiplied with: its weight, and for NVFP4 the largest of its blocks' exponents, to which
  // its blocks are brought as they are read.
  const int listed = p.plan->n_items;
  const uint32_t item0 = tid < S ? p.plan->item[tid] : 0u;   // (S <= kFewMaxSlots = NT entries)
  const uint16_t row0 = tid < S ? p.plan->row0[tid] : (uint16_t)0;
  const float weight0 = tid < S ? p.plan->weight[tid] : 0.0f;
  if (!MX && tid < S) s_top[tid] = kNoExp;
  if (tid < S) {
    s_item[tid] = item0;
    s_row0[tid] = row0;
  }
  __syncthreads();
  if (!MX) {
    for (uint32_t i = tid; i < (uint32_t)S * nch; i += kNT) {
      const uint32_t r = quotient(i, nch, p.nch_inv), c = i - r * nch;
      const uint2 e = *reinterpret_cast<const uint2*>(p.hexp + (size_t)i * 8u);
      const int used = F / 16 - (int)c * 8;
      int top = kNoExp;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e2 = (int)(int8_t)((j < 4 ? e.x : e.y) >> (8 * (j & 3)));
        top = j < used ? max(top, e2) : top;
      }
      atomicMax(&s_top[r], top);
    }
    __syncthreads();
  }
  if (tid < S) s_mul[tid] = MX ? weight0 : ldexpf(weight0, s_top[tid]);
  const int nitems = __builtin_amdgcn_readfirstlane(listed);
  __syncthreads();

  // This workgroup's part of the sequence. (Below 2^30 pairs by the limits on the sizes.)
  const uint32_t P = (uint32_t)nitems * nch, ntile = nblk / RB, Wk = P * ntile;
  uint32_t n = Wk / kDownLeast;   // workgroups that take part: not fewer than there are tiles
  n = n < ntile ? ntile : n;
  n = n < (uint32_t)p.grid ? n : (uint32_t)p.grid;
  if (blockIdx.x >= n) return;
  // (Whole tiles, the rule where little is to do, need no divisions.)
  const bool whole = n == ntile;
  const Share share(Wk, n, whole ? P : Wk / n);
  int tile = (int)blockIdx.x, q0 = 0, left = (int)P;
  if (!whole) {
    const uint32_t x0 = share.begin(blockIdx.x);
    tile = (int)(x0 / P);
    q0 = (int)(x0 - (uint32_t)tile * P);
    left = (int)(share.begin(blockIdx.x + 1) - x0);
  }

  __amdgpu_buffer_rsrc_t hr = make_rsrc(p.h, (uint32_t)S * (uint32_t)F * 2u);   // MXFP4: the item's rows
  const __amdgpu_buffer_rsrc_t er = make_rsrc(p.hexp, (uint32_t)S * nch * 8u);
  const uint32_t wrow = nch * 1024u, srow = (MX ? (nch + 15) >> 4 : (nch + 7) >> 3) * 1024u;   // of a row block
  const uint32_t lane16 = 16u * lane;
  const bool tail = (nch - 1) * kChunk + 8u * l16 >= (uint32_t)F;   // no columns in a row's last chunk
  __amdgpu_buffer_rsrc_t wr, sr;       // the tile's row blocks of the item's matrix
  uint32_t hoff = kOOB, eoff = kOOB;   // this lane's place in a row of h and of its exponents
  // MXFP4: one load holds two rows, the values in lane groups 0 and 1 and what their rounding left in
  // 2 and 3; only items of more than two tokens need another. (A load costs its instruction, also out
  // of range: two for every item take the layer of 16 tokens from 353 us to 371, one and a branch 361.)
  uint32_t hoff2 = kOOB;
  int pairs_l = 1;
  auto open_item = [&](int a) {
    const uint32_t w = (uint32_t)__builtin_amdgcn_readfirstlane((int)s_item[a]);
    wr = make_rsrc(p.codes + (size_t)(w >> 16) * wbytes + (uint32_t)tile * RB * wrow, RB * wrow);
    sr = make_rsrc(p.scales + (size_t)(w >> 16) * sbytes + (uint32_t)tile * RB * srow, RB * srow);
    const int ncol = __popc(w & 0xffffu);
    if (MX) {
      const uint32_t r0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)s_row0[a]), frow4 = (uint32_t)F * 4u;
      hr = make_rsrc(static_cast<const char*>(p.h) + (size_t)r0 * frow4, (uint32_t)ncol * frow4);
      const uint32_t at = (uint32_t)(g & 1) * frow4 + (uint32_t)(g >> 1) * (uint32_t)F * 2u + 16u * l16;
      hoff = (g & 1) < ncol ? at : kOOB;
      hoff2 = (g & 1) + 2 < ncol ? at + 2u * frow4 : kOOB;
      pairs_l = (ncol + 1) >> 1;
    } else {
      const bool in = g < ncol;
      const uint32_t hrow = (uint32_t)s_row0[a] + (uint32_t)g;
      hoff = in ? (hrow * (uint32_t)F + 8u * l16) * 2u : kOOB;
      eoff = in ? hrow * (nch * 8u) + (l16 >> 3) * 4u : kOOB;
    }
  };
  u32x4 wring[D][RB], xring[D], yring[D] = {};
  uint32_t sring[D][RB];
  uint32_t ering[D];   // the exponents of four blocks of 16 columns, the lane's own among them
  // The loads' position: item and chunk of this wave's next pair in the tile, and its steps left.
  const int da = (int)quotient(kW, nch, p.nch_inv), dc = kW - da * (int)nch;
  int a_l = 0, c_l = 0, run_l = 0;
  auto open_tile = [&](int first, int m) {   // the m pairs of the tile from pair `first` on
    run_l = wave < m ? (m - wave + kW - 1) / kW : 0;
    a_l = (int)quotient((uint32_t)(first + wave), nch, p.nch_inv);
    c_l = first + wave - a_l * (int)nch;
    open_item(run_l > 0 ? a_l : 0);   // (a wave without a pair needs a descriptor, too: its loads are out of range)
  };
  auto issue = [&](int d) {
    // (A step without a pair: as in the first launch.)
    const int in = settled_s(-run_l);   // negative: there is a pair
    const uint32_t all = (uint32_t)(in >> 31), out = kOOB & ~(uint32_t)in, c = (uint32_t)c_l;
    const uint32_t v = settled(lane16 | out), w0 = (c * 1024u) & all, s0 = scale_off<MX>(c) & all;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      wring[d][b] = ld128(wr, v, w0 + b * wrow);
      sring[d][b] = ld32(sr, v, s0 + b * srow);
    }
    const bool last = c == nch - 1;
    xring[d] = ld128(hr, settled((last && tail ? kOOB : hoff) | out), (c * 256u) & all);
    if (MX && pairs_l > 1) yring[d] = ld128(hr, settled((last && tail ? kOOB : hoff2) | out), (c * 256u) & all);
    if (!MX) ering[d] = ld32(er, settled(eoff | out), (c * 8u) & all);
    const int a0 = a_l;
    --run_l;
    c_l += dc;
    const int carry = c_l >= (int)nch ? 1 : 0;
    c_l -= carry * (int)nch;
    a_l += da + carry;
    if (a_l != a0 && run_l > 0) open_item(a_l);
  };
  bool has = false;     // the lane's token is one of the item's
  uint32_t frow = 0;    // the bytes of its row in the wave's LDS
  float mul = 0.0f;     // and what its products are multiplied with
  int pairs = 1;        // MXFP4: loads that hold the item's rows
  int top = 0;          // the exponent of the row that the lane reads (its 16-lane group's)
  auto take_item = [&](int i) {
    const uint32_t w = (uint32_t)__builtin_amdgcn_readfirstlane((int)s_item[i]);
    const uint32_t r0 = s_row0[i];
    has = (w >> l16) & 1u;
    const uint32_t fr = (uint32_t)__popc(w & ((1u << l16) - 1u)) & (kItemTok - 1);
    frow = settled((MX ? (fr & 1) + (fr >> 1) * kItemTok : fr) * kRowBytes + 64u * g);
    pairs = (__popc(w & 0xffffu) + 1) >> 1;
    mul = has ? s_mul[r0 + fr] : 0.0f;
    if (!MX) top = g < __popc(w & 0xffffu) ? s_top[r0 + g] : 0;
  };
  f32x4 tot[RB], acc[RB];
  // The item's sums into the token's: only the item's own tokens, the other columns hold
  // products that mean nothing.
  auto fold = [&]() {
#pragma unroll
    for (int b = 0; b < RB; ++b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) tot[b][i] = has ? fmaf(acc[b][i], mul, tot[b][i]) : tot[b][i];
      acc[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
  };
  unsigned char* row = s_row[wave];
  for (;;) {
    const int m = min(left, (int)P - q0);   // pairs of this tile
    left -= m;
    open_tile(q0, m);
    const int nst = run_l, turns = ((m + kW - 1) / kW + D - 1) / D;
#pragma unroll
    for (int b = 0; b < RB; ++b) tot[b] = acc[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
    int a = a_l, c = c_l;
    has = false;
    for (int turn = -1; turn < turns; ++turn) {   // turn -1 fills the ring
      // The waves go through the ring together: the CU serves its older waves first, and the
      // youngest would end up with most of its steps to do alone.
      if (turn > 0) __builtin_amdgcn_s_barrier();
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (turn >= 0) {
          // Steps past the last pair have loaded zeros and add nothing.
          const uint32_t cc = (uint32_t)c;
          if (MX) {
            *reinterpret_cast<u32x4*>(row + g * kRowBytes + 16 * l16) = xring[d];
            if (pairs > 1) *reinterpret_cast<u32x4*>(row + (kItemTok + g) * kRowBytes + 16 * l16) = yring[d];
          } else {
            const int e2 = (int)(int8_t)(ering[d] >> (4u * (l16 & 6)));
            const f16 f = (f16)ldexpf(1.0f, min(e2 - top, 0));   // (no exponent past the row's columns)
            *reinterpret_cast<f16x8*>(row + g * kRowBytes + 16 * l16) = __builtin_bit_cast(f16x8, xring[d]) * f;
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          Op bf[4], rest[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            bf[j] = *reinterpret_cast<const Op*>(row + frow + 16 * j);
            if (MX) rest[j] = *reinterpret_cast<const Op*>(row + frow + 2 * kRowBytes + 16 * j);
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            Op wf[4];
            Dec::run(wring[d][b], scale_of<MX>(sring[d][b], cc), wf);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[b] = Dec::mfma(wf[j], bf[j], acc[b]);
              if (MX) acc[b] = Dec::mfma(wf[j], rest[j], acc[b]);
            }
          }
        }
        issue(d);
        if (turn >= 0) {
          const int a0 = a;
          c += dc;
          const int carry = c >= (int)nch ? 1 : 0;
          c -= carry * (int)nch;
          a += da + carry;
          if (a != a0 && turn * D + d + 1 < nst) {   // (else the last item stays)
            fold();
            take_item(a);
          }
        }
      }
      if (turn < 0 && nst > 0) take_item(a);
    }
    fold();

    // ---- the waves' sums, then the tile or its part
#pragma unroll
    for (int b = 0; b < RB; ++b) *reinterpret_cast<f32x4*>(&s_red[wave * RB + b][l16 * 16 + 4 * g]) = tot[b];
    __syncthreads();
    // (settled: what only this part needs would be computed before the first load otherwise)
    const int per = settled_s(T) * RB * 16, at = settled_s(tile);   // values of a tile: [T][RB * 16]
    const int i0 = (int)settled((uint32_t)tid);
    const bool one = m == (int)P;   // this workgroup has all of the tile
    const Share split((uint32_t)settled_s((int)share.each), (uint32_t)settled_s((int)share.more));
    const int part0 = one ? 0 : (int)split.taker((uint32_t)at * P);
    const int parts = one ? 1 : (int)split.taker((uint32_t)at * P + P - 1) - part0 + 1;
    float* mine = p.part + ((size_t)at * p.most_parts + (blockIdx.x - part0)) * per;
    auto put = [&](int i, float v) {
      const int t = i / (RB * 16), n = i % (RB * 16);
      const size_t o = (size_t)t * p.ld_out + (size_t)at * (RB * 16) + n;
      if (p.out_bf16)
        static_cast<__bf16*>(p.out)[o] = (__bf16)v;
      else
        static_cast<float*>(p.out)[o] = v;
    };
    for (int i = i0; i < per; i += kNT) {
      const int r16 = i & 15, b = (i >> 4) % RB, t = i / (RB * 16);
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kW; ++w) v += s_red[w * RB + b][t * 16 + r16];
      if (parts == 1)
        put(i, v);
      else
        __hip_atomic_store(mine + i, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (parts > 1) {
      // Device-scope stores and loads; every wave's stores have completed (vmcnt 0) before the
      // barrier that precedes the count, and the last arriver's loads follow the barrier after it.
      __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
      __syncthreads();
      if (tid == 0)
        s_last = __hip_atomic_fetch_add(p.plan->arrived + at, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
      __syncthreads();
      if (s_last) {
        const float* base = p.part + (size_t)at * p.most_parts * per;
        for (int i = i0; i < per; i += kNT) {
          float v = 0.0f;
          for (int w = 0; w < parts; ++w)
            v += __hip_atomic_load(base + (size_t)w * per + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          put(i, v);
        }
      }
    }
    if (left == 0) break;
    __syncthreads();
    q0 = 0;
    ++tile;
  }
}

// Chunks dealt out at a time (log2): at least as many as leave every wave four or more of a tile's;
// of those the one with which the busiest CU has the fewest row block groups (more chunks at a time
// give more, smaller tiles), and of equal ones the one with the fewest tiles. sub: groups of all items.
// (6144 x 2048, one row: 192 tiles of two groups 5.3 us, 384 tiles of one 6.7. Layer of 2 tokens, 60
// experts, 2080 x 1376: 688 tiles of one group 25.5 us, 344 of two 26.4.)
int ks_log_for(int K, int64_t sub) {
  const int nch = nch_of(K);
  int l = 0;
  while (l < 4 && (nch >> (l + 1)) >= 4) ++l;
  auto most = [&](int k) {
    const int64_t tiles = ((sub << k) + kW - 1) / kW;
    return (tiles + kGrid - 1) / kGrid * (kW >> k);
  };
  int best = l;
  while (l < 4 && (1 << (l + 1)) <= nch)
    if (most(++l) < most(best)) best = l;
  return best;
}

// LDS for resident rows: what the rest leaves of a CU's 160 KB.
constexpr int kResidentBytes = 112 * 1024;
int row_lds_bytes(int K) { return nch_of(K) * 256 + 16; }
// Rows of K columns that fit.
int resident_rows(int K) { return kResidentBytes / (nch_of(K) * 256); }

// 2^32 / ppr rounded up, for pieces / ppr as the high half of a product: exact while the pieces
// (16 rows' at most, 16 ppr) times the excess (below ppr) stay under 2^32, i.e. for ppr < 2^14;
// one piece more than the last row's is never asked for.
uint32_t ppr_inverse(int K) {
  const uint32_t ppr = (uint32_t)nch_of(K) * 16u;
  return (uint32_t)(((uint64_t(1) << 32) + ppr - 1) / ppr);
}

// For quotient().
uint32_t inverse(uint32_t d) { return d == 1 ? 0xffffffffu : (uint32_t)((uint64_t(1) << 32) / d); }

template <bool MX, bool LAYER, bool FP8, bool SWIGLU, int NTOK, int D>
hipError_t launch_up(FewArgs a, int rows, int grid, hipStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto* kernel = few_up_kernel<MX, LAYER, FP8, SWIGLU, NTOK, D>;
  const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), kResidentBytes + 16 * 16, done);
  if (e != hipSuccess) return e;
  a.ppr_inv = ppr_inverse(a.K);
  a.grid = grid;
  a.grid_inv = inverse(grid);
  const int rg = kW >> a.ks_log, nsub = a.Nw / (SWIGLU ? 32 : 16);
  a.tpi_inv = inverse((nsub + rg - 1) / rg);
  kernel<<<grid, kNT, rows * row_lds_bytes(a.K), stream>>>(a);
  return hipGetLastError();
}

// Depth of the ring (chunks of a wave under way): 2, and 3 for the layer where a wave has three or more
// chunks of a tile (one token, 8 experts of 6144 x 2048: 47.1 us, 2 47.8, 4 49.1). Deeper rings bring no
// more: 16 waves' two chunks are half of what a CU can have under way, and their code is longer.
template <bool MX, bool FP8>
hipError_t launch_layer_up(const FewArgs& a, int rows, int grid, hipStream_t stream) {
  return (nch_of(a.K) - 1) >> a.ks_log < 2 ? launch_up<MX, true, FP8, true, kItemTok, 2>(a, rows, grid, stream)
                                           : launch_up<MX, true, FP8, true, kItemTok, 3>(a, rows, grid, stream);
}

template <bool MX, bool SWIGLU, int NTOK>
hipError_t launch_mv(const FewArgs& a, hipStream_t stream) {
  const int rg = kW >> a.ks_log, nsub = a.Nw / (SWIGLU ? 32 : 16), tiles = (nsub + rg - 1) / rg;
  return launch_up<MX, false, false, SWIGLU, NTOK, 2>(a, a.T, tiles < kGrid ? tiles : kGrid, stream);
}

template <bool MX, bool SWIGLU, int RB, int D>
hipError_t launch_long(FewArgs a, hipStream_t stream) {
  const int hb = SWIGLU ? RB / 2 : RB;
  const int tiles = ((SWIGLU ? a.Nw / 32 : a.Nw / 16) + hb - 1) / hb, most = 2 * kGrid;
  a.grid = tiles < most ? tiles : most;
  few_long_kernel<MX, SWIGLU, RB, D><<<a.grid, kLongNT, 0, stream>>>(a);
  return hipGetLastError();
}

template <bool MX, bool SWIGLU, int RB, int W, int D>
hipError_t launch_wide(const FewArgs& a, hipStream_t stream) {
  const int sub = SWIGLU ? a.Nw / 32 : (a.Nw / 16 + RB - 1) / RB;
  few_wide_kernel<MX, SWIGLU, RB, W, D><<<(sub + W - 1) / W, W * kWave, 0, stream>>>(a);
  return hipGetLastError();
}

template <bool MX, bool SWIGLU>
hipError_t launch_mv_rows(const FewArgs& a, hipStream_t stream) {
  // One row block a wave (two, gate and up, with SwiGLU): twice the workgroups of two a wave, which
  // bring twice the reads under way: 2048 x 6144, one row 9.0 -> 6.9 us, 16384 x 6144 16.1 -> 14.8,
  // 2048 x 2048, 16 rows 9.0 -> 7.3; slower only at 32768 x 1024 (7.9 -> 8.1).
  constexpr int RB = SWIGLU ? 2 : 1;
  if (a.T <= resident_rows(a.K))
    return a.T > 4 ? launch_mv<MX, SWIGLU, 16>(a, stream) : launch_mv<MX, SWIGLU, 4>(a, stream);
  // Rows past the resident ones' LDS. More tiles than few_long_kernel has workgroups: the kernel
  // whose waves share the rows. T = 16, K = 6144, cold weights, few_long / few_wide, us:
  //   weight rows       8192        16384       24576       32768       65536       152064
  //   NVFP4          12.6 / 23.1  21.3 / 24.9 36.9 / 26.9 38.0 / 28.6 71.2 / 50.6  165 / 119
  //   MXFP4           9.0 / 16.3  17.7 / 19.6 30.9 / 22.7 33.3 / 24.5 60.6 / 45.7  141 / 106
  //   SWIGLU, NVFP4  12.0 / 34.2  20.3 / 36.6 35.2 / 39.1 36.3 / 41.5 67.8 / 49.8  163 / 122
  // few_long_kernel with one row block a wave (two chunks under way) while that finds every
  // workgroup a CU of its own: 2048 rows 9.8, against 11.5 with two; from there on two (one chunk).
  const int tiles = SWIGLU ? a.Nw / 64 : a.Nw / 32;
  if (tiles > 512) return launch_wide<MX, SWIGLU, RB, 8, 4>(a, stream);
  if constexpr (!SWIGLU)
    if (a.Nw / 16 <= kGrid) return launch_long<MX, SWIGLU, 1, 2>(a, stream);
  return launch_long<MX, SWIGLU, 2, 1>(a, stream);
}

}  // namespace

// One row block a tile where such tiles, uncut, find a CU each and are short (at most 512 pairs a CU):
// twice the CUs of two a tile. Layers with cold weights, one / two blocks, us: 2048 x 1024 with 8 / 64 /
// 128 rows 18.3 / 21.6, 42.5 / 49.9, 53.0 / 57.6; 4096 x 2048 with 8 / 32 / 64 / 128 rows (128, 512, 1024,
// 2048 pairs) 35.3 / 40.5, 85 / 85.5, 129 / 123, 177 / 161: two blocks read each row of h half as often.
int few_down_blocks(int T, int k, int Nw, int K) {
  return Nw / 16 <= kGrid && (int64_t)T * k * nch_of(K) * (Nw / 16) <= 512 * kGrid ? 1 : 2;
}
int few_down_workgroups(int T, int k, int Nw, int K) {
  const int64_t ntile = Nw / (16 * few_down_blocks(T, k, Nw, K)), most = (int64_t)T * k * nch_of(K) * ntile / kDownLeast;
  const int64_t n = most > ntile ? most : ntile;
  return n < kGrid ? (int)n : kGrid;
}
int few_down_parts(int T, int k, int Nw, int K) {
  // A tile of P pairs holds at most ceil(P n / W) + 1 of the n workgroups' parts, and P / W = 1 / ntile
  const int ntile = Nw / (16 * few_down_blocks(T, k, Nw, K));
  return (few_down_workgroups(T, k, Nw, K) + ntile - 1) / ntile + 1;
}

hipError_t launch_few_matvec(FewArgs a, bool mx, bool swiglu, hipStream_t stream) {
  a.ks_log = ks_log_for(a.K, swiglu ? a.Nw / 32 : a.Nw / 16);
  if (mx) return swiglu ? launch_mv_rows<true, true>(a, stream) : launch_mv_rows<true, false>(a, stream);
  return swiglu ? launch_mv_rows<false, true>(a, stream) : launch_mv_rows<false, false>(a, stream);
}

hipError_t launch_few_layer(FewArgs up, FewArgs down, bool mx, hipStream_t stream) {
  up.ks_log = ks_log_for(up.K, (int64_t)up.T * up.k * (up.Nw / 32));
  const int fit = resident_rows(up.K);   // >= 1 by the limit on H
  up.item_tok = fit < kItemTok ? fit : kItemTok;
  const int rg = kW >> up.ks_log, nsub = up.Nw / 32;
  const int64_t tiles = (int64_t)up.T * up.k * ((nsub + rg - 1) / rg);   // bound: every slot an item
  const int grid = tiles < kGrid ? (int)tiles : kGrid;
  const int rows = up.T < up.item_tok ? up.T : up.item_tok;
  const hipError_t e = mx       ? launch_layer_up<true, false>(up, rows, grid, stream)
                       : up.fp8 ? launch_layer_up<false, true>(up, rows, grid, stream)
                                : launch_layer_up<false, false>(up, rows, grid, stream);
  if (e != hipSuccess) return e;
  const int wgs = few_down_workgroups(down.T, down.k, down.Nw, down.K);
  down.nch_inv = inverse((uint32_t)nch_of(down.K));
  down.grid = wgs;
  const bool two = few_down_blocks(down.T, down.k, down.Nw, down.K) == 2;
  auto* kernel = mx ? (two ? few_down_kernel<true, 2> : few_down_kernel<true, 1>)
                    : (two ? few_down_kernel<false, 2> : few_down_kernel<false, 1>);
  kernel<<<wgs, kNT, 0, stream>>>(down);
  return hipGetLastError();
}

}  // namespace nvfp4moe
