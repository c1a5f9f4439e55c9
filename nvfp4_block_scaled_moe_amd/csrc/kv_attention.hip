// Attention of many new tokens over the paged cache (gfx950): prompts, chunks of prompts, and batches
// that mix them with sequences that decode; and the choice between this and kv_attention_few.hip.
//   out[t, h] = sum_j softmax_j(scale q[t, h] . k[j, h / G]) v[j, h / G]   over the keys j that t sees
//
// Bound by the matrix cores (4 D flops for each pair of row and key) and, beside them, by the
// exponentials: 32 x 32 scores take 64 D / 8 matrix cycles for both products and about 500 vector
// cycles, so that two waves a SIMD keep both busy. A tile is 128 or 256 rows (token, head of the group) of
// one key head, 32 a wave; keys and values of 64 tokens at a time lie in LDS, twice, and are
// requested one block ahead (bf16: straight into LDS; E4M3: through registers, where keys become bf16 and
// values f16, which hold them exactly). Scores are transposed, S^T = K Q^T: a lane holds the scores of
// one row, and with K's rows in LDS in the right order these are, after the exponential, the operand
// of O^T = V^T P^T without another move. The rows of LDS are not padded; their 16-byte words are
// permuted by the row, so that reads have no bank conflicts. Blocks that every row of a tile sees go half a block
// at a time through three stages that do not wait for each other (below); the others, at the diagonal and a
// window's start, are masked and taken one after another.
//
// 2048 tokens over 14000 keys, 64 heads over 8, bf16: D 128 915 to 991 us by card, 1.02 to 1.10 PFLOP/s (a large
// matrix product reaches 1.42), D 64 600 us (0.84: twice the exponentials for a flop); E4M3 2 to 5% more. 32 heads
// of 96 / 160 / 192 / 224 / 256 over 6000: 0.85 / 0.69 / 0.67 / 0.65 / 0.70 PFLOP/s (one wave a SIMD from D 160 on:
// the outputs fill the registers). The matrix cores are busy half of the time at a clock that the power limit holds
// at 1.9 GHz. Copies with a part left out: without the requests 15% less time, without exponentials 12%, without the
// reads of V from LDS 8%.
//
// Weights of the second product are exponentials rounded to bf16 (about as much again as the rounding of the
// output; two bf16 values each would cost half the second product again) or, with an E4M3 cache, to f16. Their
// sum is taken before that rounding. The running maximum is moved only when scores are far above it: until then
// weights above 1 keep their relative precision.
//
// The work is divided as Division says; where a tile is split, its parts leave unnormalised sums, which a
// second launch joins.
#include <type_traits>

#include "gemm_common.h"
#include "kv_attention.h"

namespace nvfp4moe {

namespace {

constexpr float kSlack = 8.0f;        // base 2 logits by which a score may exceed the running maximum,
constexpr float kHigh = 32768.0f;     // and, where that is looked at by the sums alone, sum of 16 weights (2^15)
constexpr int kBlockLog = kChunkBlockLog, kBlock = 1 << kBlockLog;   // keys of a block
template <int W>
struct OfWaves {
  static constexpr Division kDivision = chunk_division(W);
};

// 16 bytes a lane straight into LDS (lane l at lds + 16 l), from global memory or from a buffer (whose base
// and offset `soff` are the wave's: no address arithmetic in the lanes).
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void dma16(const char* from, char* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

// max (or sum) of a lane's value and that of the lane 32 away
__device__ __forceinline__ float max_across(float v) {
  const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Numbers of the second product: bf16 as the cache holds them, or f16 for E4M3, which f16 holds as exactly and whose
// weights then have 11 bits instead of 8. f16 ends at 65504 and, below, at 2^-24: weights are taken times 2^kRaise,
// which leaves kSlack above, and below the maximum 2^-31 (a million keys of less are together less than 2^-11).
template <bool F16>
struct Second {
  typedef __bf16 T;
  typedef bf16x8 V;
  static constexpr float kRaise = 0.0f;
  static constexpr uint32_t kExponent = 0x7f807f80u, kOne = 0x00800080u;
  static __device__ __forceinline__ f32x16 product(V a, V b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
};
template <>
struct Second<true> {
  typedef _Float16 T;
  typedef f16x8 V;
  static constexpr float kRaise = 7.0f;
  static constexpr uint32_t kExponent = 0x7c007c00u, kOne = 0x04000400u;
  static __device__ __forceinline__ f32x16 product(V a, V b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
};
// Bit 15 and 31: those of two such numbers (a word) that are NaN or Inf.
template <bool F16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & Second<F16>::kExponent) + Second<F16>::kOne) & 0x80008000u;
}
// All 16 bits of each of those.
__device__ __forceinline__ uint32_t halves_of(uint32_t bits) { return (bits >> 15) * 0xffffu; }

template <int D, bool FP8>
struct Chunk {
  static constexpr int kWords = D / 8;               // 16-byte words of a key in LDS
  static constexpr int kBytes = kBlock * D * 2;      // of a block's keys, and of its values
  static constexpr int kSteps = D / 16;              // of the first product
  static constexpr int kDTiles = D / 32;             // of the second
  // (E4M3 of D 256: the words on their way leave no registers for two halves' scores; 752 us, 809 pipelined, for 2048
  // new tokens over 6000; bf16 696 pipelined, 820 not)
  static constexpr bool kPipelined = !FP8 || D <= 224;
  // LDS serves 16 lanes' 16-byte words a cycle where they lie in different 16ths of its 256-byte lines. A
  // product reads one word of 16 rows at once, so word w of row r lies at w ^ swizzle(r): the rows' own
  // places in the lines (kWords 16ths apart) and the swizzle make 16 different ones.
  static __device__ __forceinline__ int swizzle(int r) {
    return kWords % 16 == 0 ? r % 16 : kWords % 8 == 0 ? r / 2 % 8 : r / 4 % 4;
  }
  static __device__ __forceinline__ int v_swizzle(int d) { return d / 2 % 8; }   // rows of V^T have 8 words
};

// Key, of 16, of K's row r in LDS: row 8x + 4y + z holds key 8y + 4x + z, so that the scores of a lane
// (rows 8 (i / 4) + 4 half + i % 4) are those of 8 consecutive keys.
__device__ __forceinline__ int key_of_row(int r) { return r / 4 % 2 * 8 + r / 8 * 4 + r % 4; }

template <int D, bool FP8, int W>
__global__ __launch_bounds__(W* kWave, D > 128 ? 1 : 2) void chunk_kernel(const KvAttnArgs p) {
  using C = Chunk<D, FP8>;
  using S2 = Second<FP8>;
  constexpr Division kDivision = chunk_division(W);
  constexpr int kRows = kDivision.tile_rows();
  extern __shared__ __attribute__((aligned(16))) char smem[];   // two of: keys [64, D], values [D, 64]; then
  uint32_t* s_any = reinterpret_cast<uint32_t*>(smem + 4 * Chunk<D, FP8>::kBytes);   // a flag a wave
  const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane % 32, half = lane / 32;
  const int h = blockIdx.x % p.Hkv;
  const Segment sg = segment_of<false>(p, kDivision, blockIdx.x / p.Hkv);
  if (!sg.found) return;
  const CacheBatchArgs& b = p.batch;
  const Sequence& seq = sg.seq;

  // This lane's row, and the keys that it sees; those that all rows of the tile see; those that any of this
  // wave's rows sees.
  const int rows = seq.n * p.G, row0 = sg.tile * kRows + 32 * wave;
  const int row = min(row0 + col, rows - 1), token = row / p.G, head = h * p.G + row - token * p.G;
  const Seen mine = seen_by(seq.position(token), p.window, seq.cap);
  auto seen_of = [&](int r) __attribute__((always_inline)) { return seen_by(seq.position(min(r, rows - 1) / p.G), p.window, seq.cap); };
  const int all_lo = seen_of(sg.tile * kRows + kRows - 1).lo, all_hi = seen_of(sg.tile * kRows).hi;
  const int any_lo = seen_of(row0).lo, any_hi = row0 < rows ? seen_of(row0 + 31).hi : 0;

  bf16x8 q[C::kSteps];
  {
    const uint16_t* from = p.q + (seq.row0 + token) * p.q_row + head * p.q_head + 8 * half;
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i) q[i] = *reinterpret_cast<const bf16x8*>(from + 16 * i);
  }
  const float log2_scale = p.scale * kLog2e * (FP8 && p.k_scale ? p.k_scale[h] : 1.0f);

  // Staging: a block's keys and V^T in loads of a wave, dealt to the waves in order. A load of keys is of 16 keys
  // (one page's: pages are whole multiples of 16), of V^T 8 rows (E4M3: 16), of which a lane takes 16 bytes.
  constexpr int kSize = FP8 ? 1 : 2;
  const int page = b.page, page_mask = page - 1;
  const int64_t head_bytes = (int64_t)page * D * kSize;
  const int* table = b.page_table + sg.s * b.ld_table;
  // (bf16: a load is 8 rows of V^T, whose swizzle is the lane's and, in every second load, 4: the lane's word
  // is then one of the block's other half)
  const int v_word = FP8 ? lane % 4 : (lane % 8) ^ (lane / 16);       // of the 4 or 8 words of a row of V^T
  const int v_key = FP8 ? 16 * v_word : 8 * v_word, v_row = FP8 ? lane / 4 : lane / 8;
  constexpr int kKParts = FP8 ? (D + 63) / 64 : D / 32;                         // loads of 16 keys
  constexpr int kKAll = 4 * kKParts, kKLoads = (kKAll + W - 1) / W;             // of a block; of a wave
  constexpr int kVRows = FP8 ? 16 : 8, kVAll = D / kVRows, kVLoads = (kVAll + W - 1) / W;
  const int k_load0 = wave * kKLoads, v_load0 = wave * kVLoads;
  struct Pages {
    int k[kKLoads], v, v2;   // of this wave's loads of keys; of this lane's values, in the two kinds of load
  };
  const bool whole = b.page_log >= kBlockLog;   // a block lies in one page
  auto pages_of = [&](int block) __attribute__((always_inline)) {
    const int key = block << kBlockLog;
    Pages r;
    if (whole) {
      const int c = key >> b.page_log, at = c < b.cols ? ld_const(table, c) : -1;
#pragma unroll
      for (int j = 0; j < kKLoads; ++j) r.k[j] = at;
      r.v = r.v2 = at;
    } else {
#pragma unroll
      for (int j = 0; j < kKLoads; ++j) {
        const int kc = (key + (k_load0 + j) / kKParts * 16) >> b.page_log;
        r.k[j] = kc < b.cols ? ld_const(table, kc) : -1;
      }
      const int vc = (key + v_key) >> b.page_log, vc2 = (key + (v_key ^ 32)) >> b.page_log;
      r.v = vc < b.cols ? table[vc] : -1;
      r.v2 = FP8 ? -1 : vc2 < b.cols ? table[vc2] : -1;
    }
    return r;
  };
  u32x4v raw_k[FP8 ? kKLoads : 1], raw_v[FP8 ? kVLoads : 1];
  uint32_t k_off[kKLoads];   // this lane's words among a load's 16 keys: bytes from the first key
#pragma unroll
  for (int j = 0; j < kKLoads; ++j) {
    const int i = (k_load0 + j) % kKParts * 64 + lane;
    if (FP8) {
      k_off[j] = i < D ? i / (D / 16) * D + i % (D / 16) * 16 : kOOB;
    } else {
      const int r = i / C::kWords;
      k_off[j] = key_of_row(r) * (2 * D) + ((i % C::kWords) ^ C::swizzle(r)) * 16;
    }
  }
  const uint32_t v_off = (uint32_t)((v_row * page + (whole ? v_key : v_key & page_mask)) * kSize);
  // Requests a block's keys or values (bf16: into LDS buffer `to`; E4M3: into registers).
  auto request_k = [&](int block, const Pages& pg, char* to) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kKLoads; ++j) {
      const int n = k_load0 + j, g = n / kKParts;
      if (kKAll % W != 0 && n >= kKAll) break;
      const int at = whole ? pg.k[0] : pg.k[j];
      const bool ok = at >= 0 && at < b.pages;
      const __amdgpu_buffer_rsrc_t k =
          make_rsrc(static_cast<const char*>(p.k_cache) + ((int64_t)(ok ? at : 0) * p.Hkv + h) * head_bytes, (uint32_t)head_bytes);
      const uint32_t first = (uint32_t)(((block << kBlockLog) + 16 * g) & page_mask) * (D * kSize);
      if constexpr (FP8)
        raw_k[j] = __builtin_amdgcn_raw_buffer_load_b128(k, k_off[j], first, 0);
      else
        dma16(k, to + g * 32 * D + n % kKParts * 1024, k_off[j], first);
    }
  };
  // (and says which of the block's 16s of keys have no page, a bit each)
  auto request_v = [&](int block, const Pages& pg, char* to) __attribute__((always_inline)) {
    const int key = block << kBlockLog;
    const bool v_ok = pg.v >= 0 && pg.v < b.pages;
    if (whole) {
      const __amdgpu_buffer_rsrc_t v = make_rsrc(
          static_cast<const char*>(p.v_cache) + ((int64_t)(v_ok ? pg.k[0] : 0) * p.Hkv + h) * head_bytes, (uint32_t)head_bytes);
      const uint32_t v_first = (uint32_t)(key & page_mask) * kSize;
#pragma unroll
      for (int j = 0; j < kVLoads; ++j) {
        const int d = (v_load0 + j) * kVRows;
        if (kVAll % W != 0 && d >= D) break;
        if constexpr (FP8)
          raw_v[j] = __builtin_amdgcn_raw_buffer_load_b128(v, v_off, v_first + (uint32_t)(d * page), 0);
        else
          dma16(v, to + C::kBytes + d * 128, d / 8 % 2 ? v_off ^ 64u : v_off, v_first + (uint32_t)(d * page) * 2);
      }
    } else {   // (pages of 16 and 32: 32 keys on, a lane's place in its page is the same)
      const bool v2_ok = pg.v2 >= 0 && pg.v2 < b.pages;
      const char* v = static_cast<const char*>(p.v_cache) + ((int64_t)(v_ok ? pg.v : 0) * p.Hkv + h) * head_bytes + v_off;
      const char* v2 = static_cast<const char*>(p.v_cache) + ((int64_t)(v2_ok ? pg.v2 : 0) * p.Hkv + h) * head_bytes + v_off;
#pragma unroll
      for (int j = 0; j < kVLoads; ++j) {
        const int d = (v_load0 + j) * kVRows;
        if (kVAll % W != 0 && d >= D) break;
        if constexpr (FP8) {
          raw_v[j] = *reinterpret_cast<const u32x4v*>(v + (int64_t)d * page);
        } else {
          dma16((d / 8 % 2 ? v2 : v) + (int64_t)d * page * 2, to + C::kBytes + d * 128);
        }
      }
    }
    const uint64_t bad = __ballot(!v_ok);   // (lanes of the first row of V^T: of each 16 keys one)
    return FP8 ? (uint32_t)(bad & 15u) : (uint32_t)((bad & 1u) | (bad >> 1 & 2u) | (bad >> 2 & 4u) | (bad >> 3 & 8u));
  };
  // E4M3: what they brought, keys as bf16 and values as f16, into LDS.
  auto put_k = [&](char* at0, char* at1, const u32x4v& w) __attribute__((always_inline)) {
    *reinterpret_cast<bf16x8*>(at0) = e4m3x8_to_bf16(w[0], w[1]);
    *reinterpret_cast<bf16x8*>(at1) = e4m3x8_to_bf16(w[2], w[3]);
  };
  auto put_v = [&](char* at0, char* at1, const u32x4v& w) __attribute__((always_inline)) {
    *reinterpret_cast<f16x8*>(at0) = e4m3x8_to_f16(w[0], w[1]);
    *reinterpret_cast<f16x8*>(at1) = e4m3x8_to_f16(w[2], w[3]);
  };
  auto place_k = [&](char* to) __attribute__((always_inline)) {
    if constexpr (FP8) {
#pragma unroll
      for (int j = 0; j < kKLoads; ++j) {
        const int n = k_load0 + j, i = n % kKParts * 64 + lane;
        if (kKAll % W != 0 && n >= kKAll) break;
        const int r = key_of_row(i / (D / 16)), w = i % (D / 16) * 2;   // (key_of_row is its own inverse)
        char* line = to + (n / kKParts * 16 + r) * (2 * D);
        if (D % 64 == 0 || i < D) put_k(line + (w ^ C::swizzle(r)) * 16, line + ((w + 1) ^ C::swizzle(r)) * 16, raw_k[j]);
      }
    }
  };
  auto place_v = [&](char* to) __attribute__((always_inline)) {
    if constexpr (FP8) {
#pragma unroll
      for (int j = 0; j < kVLoads; ++j) {
        const int d = (v_load0 + j) * 16 + v_row, x = C::v_swizzle(d);
        if (kVAll % W != 0 && (v_load0 + j) * 16 >= D) break;
        char* line = to + C::kBytes + d * 128;
        put_v(line + ((2 * v_word) ^ x) * 16, line + ((2 * v_word + 1) ^ x) * 16, raw_v[j]);
      }
    }
  };
  // Every wave's words are in LDS (and, direct ones, waited for).
  auto arrive = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    __syncthreads();
  };

  // base: what exponentials are taken from. Before any score above -Inf it lies so far down that the first one shows
  // in the sums (and -Inf less it is still -Inf: a weight of 0).
  constexpr float kNone = -3e38f;
  float m = -INFINITY, base = kNone, l = 0.0f;
  f32x16 o[C::kDTiles];
  uint32_t lost[(C::kDTiles + 1) / 2] = {};   // bit 16 (d % 2) + i: o[d][i] is to be NaN
#pragma unroll
  for (int d = 0; d < C::kDTiles; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;

  // The pieces of a step, for half a block (32 keys): scores; their exponentials as weights of the second product;
  // that product. Score i of tile a: key 32a + 16 (i / 8) + 8 half + i % 8 of the block.
  struct Weights {
    typename S2::V w[2];
  };
  auto score_step = [&](const char* in, int a, int i, const f32x16& s) __attribute__((always_inline)) {
    const bf16x8 k = *reinterpret_cast<const bf16x8*>(in + (32 * a + col) * (2 * D) + ((2 * i + half) ^ C::swizzle(col)) * 16);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[i], s, 0, 0, 0);
  };
  auto scores = [&](const char* in, int a, f32x16& s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i) s = score_step(in, a, i, s);
  };
  auto exponentials = [&](const f32x16& s, Weights& w, float& sum) __attribute__((always_inline)) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], log2_scale, -base));
      sum += e;
      w.w[i / 8][i % 8] = (typename S2::T)e;
    }
  };
  auto values = [&](const char* in, int a, const Weights& w) __attribute__((always_inline)) {
    const char* rows_at = in + C::kBytes + col * 128;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int d = 0; d < C::kDTiles; ++d) {
        const typename S2::V v =
            *reinterpret_cast<const typename S2::V*>(rows_at + d * 4096 + ((4 * a + 2 * u + half) ^ C::v_swizzle(col)) * 16);
        o[d] = S2::product(v, w.w[u], o[d]);
      }
  };
  // Largest score of each row, times the scale.
  auto largest = [&](const f32x16& s) __attribute__((always_inline)) {
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
    return max_across(top) * log2_scale;
  };
  // The row's maximum moves to `next`.
  auto move_maximum = [&](float next) __attribute__((always_inline)) {
    const float shrink = next == m ? 1.0f : __builtin_amdgcn_exp2f(m - next);
    m = next;
    base = m == -INFINITY ? kNone : m - S2::kRaise;
    l *= shrink;
#pragma unroll
    for (int d = 0; d < C::kDTiles; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] *= shrink;
  };

  // A block in LDS; EDGE: with keys that some row of the tile does not see.
  auto use = [&](auto edge, int block, const char* in, uint32_t bad_pages) __attribute__((always_inline)) {
    constexpr bool EDGE = decltype(edge)::value;
    const int begin = block << kBlockLog;
    if (row0 >= rows) return;                                            // this wave has no rows: it brings words alone
    if (EDGE && (begin >= any_hi || begin + kBlock <= any_lo)) return;   // none that its rows see
    if (bad_pages != 0u) {   // (a page holds 16 keys or more) a row that sees one of a page that is none
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if ((bad_pages >> g & 1u) && mine.lo < begin + 16 * g + 16 && mine.hi > begin + 16 * g) l = NAN;
    }
    const uint32_t from_lo = (uint32_t)(begin + 8 * half - mine.lo), seen = (uint32_t)max(mine.hi - mine.lo, 0);
    f32x16 s[2];
    Weights w[2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[a][i] = 0.0f;
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i)
#pragma unroll
      for (int a = 0; a < 2; ++a) s[a] = score_step(in, a, i, s[a]);
    if constexpr (EDGE) {
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[a][i] = from_lo + (uint32_t)(32 * a + 16 * (i / 8) + i % 8) < seen ? s[a][i] : -INFINITY;
    }
    const float top = fmaxf(largest(s[0]), largest(s[1]));
    if (__any(top > m + kSlack)) move_maximum(top > m + kSlack ? top : m);
    float sum[2];
#pragma unroll
    for (int a = 0; a < 2; ++a) exponentials(s[a], w[a], sum[a]);
    l += sum[0] + sum[1];
#pragma unroll
    for (int a = 0; a < 2; ++a) values(in, a, w[a]);
  };

  // Values that some row does not see (or no row: what a page holds behind its last token) must not reach it,
  // NaN and Inf included, which a zero weight does not hold back. Where a block with such keys has any: zeros in
  // their place, and the dims that they spoil in the rows that see them are kept as bits, for the end. (Each wave looks at its part of V^T.)
  auto clean = [&](int block, char* in) __attribute__((always_inline)) {
    constexpr int kCleanLoads = D / (8 * W);
    static_assert(D % (8 * W) == 0, "waves share V^T evenly");
    uint32_t any = 0u;
    char* mine_v = in + C::kBytes + wave * (C::kBytes / W) + lane * 16;
#pragma unroll
    for (int i = 0; i < kCleanLoads; ++i) {
      const u32x4v v = *reinterpret_cast<const u32x4v*>(mine_v + 1024 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) any |= not_finite<FP8>(v[j]);
    }
    if (lane == 0) s_any[wave] = 0u;
    if (__any(any != 0u) && lane == 0) s_any[wave] = 1u;
    __syncthreads();
    any = 0u;
#pragma unroll
    for (int i = 0; i < W; ++i) any |= s_any[i];
    if (any == 0u) return;
    const uint32_t from_lo = (uint32_t)((block << kBlockLog) + 8 * half - mine.lo), seen = (uint32_t)max(mine.hi - mine.lo, 0);
#pragma unroll 1
    for (int u = 0; u < 4; ++u) {
      bf16x8 sees;
#pragma unroll
      for (int i = 0; i < 8; ++i) sees[i] = from_lo + (uint32_t)(16 * u + i) < seen ? (__bf16)1.0f : (__bf16)0.0f;
#pragma unroll
      for (int d = 0; d < C::kDTiles; ++d) {
        u32x4v bad = *reinterpret_cast<const u32x4v*>(in + C::kBytes + (32 * d + col) * 128 + ((2 * u + half) ^ C::v_swizzle(col)) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) bad[i] = halves_of(not_finite<FP8>(bad[i])) & 0x3f803f80u;   // a bf16 1 for each
        f32x16 n;   // how many of them each row sees
#pragma unroll
        for (int i = 0; i < 16; ++i) n[i] = 0.0f;
        n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, bad), sees, n, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 16; ++i) lost[d / 2] |= n[i] > 0.0f ? 1u << (16 * (d % 2) + i) : 0u;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < kCleanLoads; ++i) {
      u32x4v v = *reinterpret_cast<const u32x4v*>(mine_v + 1024 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] &= ~halves_of(not_finite<FP8>(v[j]));
      *reinterpret_cast<u32x4v*>(mine_v + 1024 * i) = v;
    }
    __syncthreads();
  };

  if (sg.blocks > 0) {
    const int end = sg.block0 + sg.blocks;
    // The blocks of which every row of the tile sees all keys, [lead, full), and those before and behind them.
    const int lead = min(max((all_lo + kBlock - 1) >> kBlockLog, sg.block0), end), full = min(max(all_hi >> kBlockLog, lead), end);
    char* now = smem;                     // the block in use
    char* then = smem + 2 * C::kBytes;    // the next one
    int block = sg.block0;
    auto ahead = [&](int i) __attribute__((always_inline)) { return min(i, end - 1); };
    Pages pg = pages_of(block);
    request_k(block, pg, now);
    uint32_t bad = request_v(block, pg, now);
    pg = pages_of(ahead(block + 1));
    place_k(now);
    place_v(now);
    arrive();
    auto step = [&](auto edge) __attribute__((always_inline)) {
      uint32_t next_bad = 0u;
      if (block + 1 < end) {
        request_k(block + 1, pg, then);
        next_bad = request_v(block + 1, pg, then);
        pg = pages_of(ahead(block + 2));
      }
      if constexpr (decltype(edge)::value) clean(block, now);
      use(edge, block, now, bad);
      if (block + 1 < end) {
        place_k(then);
        place_v(then);
      }
      arrive();
      char* t = now;
      now = then;
      then = t;
      bad = next_bad;
      ++block;
    };
    while (block < lead) step(std::true_type{});
    if constexpr (!C::kPipelined) {
      while (block < full) step(std::false_type{});
    } else if (block < full) {
      // Half a block at a time, in one stretch of code without branches: the scores of the next half, the
      // exponentials of this one and the second product of the one before, which do not wait for each other, so
      // that the matrix cores work while the exponentials are taken. Keys run a block ahead of values: K of the
      // block two on is requested with V of the next one. The maximum stays, unless the sum of a half's
      // exponentials shows that scores are far above it; then these are taken again.
      uint32_t missing = bad;   // any key without a page: every row sees it
      Pages pg2 = pages_of(ahead(block + 2));
      if (block + 1 < end) request_k(block + 1, pg, then);
      auto turn = [&]() __attribute__((always_inline)) {
        char* t = now;
        now = then;
        then = t;
      };
      auto bring = [&]() __attribute__((always_inline)) {   // V of the next block, K of the one after it
        bad = request_v(block + 1, pg, then);
        missing |= bad;
        if (block + 2 < end) request_k(block + 2, pg2, now);
        pg = pg2;
        pg2 = pages_of(ahead(block + 3));
      };
      auto have = [&]() __attribute__((always_inline)) {
        place_v(then);
        if (block + 2 < end) place_k(now);
        arrive();
        turn();
        ++block;
      };
      auto bring_last = [&]() __attribute__((always_inline)) {   // (what follows brings its keys with its values)
        if (block + 1 < end) bad = request_v(block + 1, pg, then);
      };
      auto have_last = [&]() __attribute__((always_inline)) {
        if (block + 1 < end) place_v(then);
        arrive();
        pg = pg2;
        turn();
        ++block;
      };
      if (row0 < rows) {
        f32x16 s0, s1;
        Weights w0, w1;
        float sum;
        auto settle = [&](const f32x16& s, Weights& w) __attribute__((always_inline)) {
          if (__any(sum > kHigh)) {
            // (a row's maximum moves by its own scores alone, so that no row's bits depend on another's)
            const float top = largest(s);
            move_maximum(max_across(sum) > kHigh ? top : m);
            exponentials(s, w, sum);
          }
          l += sum;
        };
        // from s1, the scores of the second half of `block`, and w0, the weights of its first, to the next block's
        auto advance = [&]() __attribute__((always_inline)) {
          bring();
          scores(then, 0, s0);
          exponentials(s1, w1, sum);
          values(now, 0, w0);
          settle(s1, w1);
          scores(then, 1, s1);
          exponentials(s0, w0, sum);
          values(now, 1, w1);
          settle(s0, w0);
          have();
        };
        scores(now, 0, s0);
        const float top = largest(s0);
        if (__any(top > m + kSlack)) move_maximum(top > m + kSlack ? top : m);
        scores(now, 1, s1);
        exponentials(s0, w0, sum);
        settle(s0, w0);
        if (block + 1 < end) place_k(then);
        arrive();
        while (block + 1 < full) advance();
        bring_last();
        exponentials(s1, w1, sum);
        values(now, 0, w0);
        settle(s1, w1);
        values(now, 1, w1);
        have_last();
      } else {   // a wave without rows brings words alone
        if (block + 1 < end) place_k(then);
        arrive();
        while (block + 1 < full) {
          bring();
          have();
        }
        bring_last();
        have_last();
      }
      if (missing != 0u) l = NAN;
    }
    while (block < end) step(std::true_type{});
  }
  {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  uint32_t any_lost = 0u;
#pragma unroll
  for (int d = 0; d < (C::kDTiles + 1) / 2; ++d) any_lost |= lost[d];
  if (any_lost != 0u) {
#pragma unroll
    for (int d = 0; d < C::kDTiles; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = lost[d / 2] >> (16 * (d % 2) + i) & 1u ? NAN : o[d][i];
  }
  if (row0 + col >= rows) return;
  // this lane: dims 32 d + 8 (i / 4) + 4 half + i % 4 of its row
  if (sg.parts > 1) {
    const Sums part(p, kDivision, sg.slot, h);
    const int r = 32 * wave + col;
#pragma unroll
    for (int d = 0; d < C::kDTiles; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(part.o + r * D + 32 * d + 2 * i + 4 * half) = make_float4(o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]);
    if (half == 0) {
      part.ml[2 * r] = m;
      part.ml[2 * r + 1] = l;
    }
  } else {
    const float f = normalize(seq, token, l, FP8 && p.v_scale ? p.v_scale[h] : 1.0f);
    uint16_t* to = p.out + (seq.row0 + token) * p.o_row + head * p.o_head + 4 * half;
#pragma unroll
    for (int d = 0; d < C::kDTiles; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<uint2*>(to + 32 * d + 2 * i) =
            make_uint2(bf16x2(o[d][i] * f, o[d][i + 1] * f), bf16x2(o[d][i + 2] * f, o[d][i + 3] * f));
  }
}

template <int D, bool FP8, int W>
hipError_t launch(const KvAttnArgs& a, hipStream_t stream) {
  constexpr int lds = 4 * Chunk<D, FP8>::kBytes + W * 4;
  static std::atomic<uint64_t> done{0};
  if (lds > 65536) {
    const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(chunk_kernel<D, FP8, W>), lds, done);
    if (e != hipSuccess) return e;
  }
  const int64_t groups = chunk_division(W).segments(a.batch.T, a.batch.B, a.Hkv, a.G) * a.Hkv;
  chunk_kernel<D, FP8, W><<<dim3((unsigned)groups), W * kWave, lds, stream>>>(a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_join<FP8, OfWaves<W>>(a, stream);
}

// Waves of a workgroup. 8 for D 128 (D 64 has three waves a SIMD with W 4: 614 us, 657 with 8), where sequences have
// rows for whole tiles of 256, on average, and the page table has columns for keys enough that what these bring is most
// of the time: 2048 new tokens over 14000 keys 930 us, 995 with 4, 128 over 30000 139 and 149; but 8 prompts of 1024
// tokens 222, 215 with 4. What a sequence has of those keys, and what a window leaves of them, is not looked at: these
// prompts in a table of 33000 tokens take 215, 206 with 4, and the first case with a window of 1000 103, 97 with 4.
bool many_rows(int T, int B, int G, int D) { return D == 128 && (int64_t)T * G >= (int64_t)1024 * B; }
int waves_of(const KvAttnArgs& a) {
  return many_rows(a.batch.T, a.batch.B, a.G, a.D) && (int64_t)a.batch.cols << a.batch.page_log >= 4096 ? 8 : 4;
}

template <int D, bool FP8>
hipError_t launch_w(const KvAttnArgs& a, hipStream_t stream) {
  if constexpr (D == 128) {
    if (waves_of(a) == 8) return launch<D, FP8, 8>(a, stream);
  }
  return launch<D, FP8, 4>(a, stream);
}

template <bool FP8>
hipError_t launch_d(const KvAttnArgs& a, hipStream_t stream) {
  switch (a.D / 32) {
    case 1: return launch_w<32, FP8>(a, stream);
    case 2: return launch_w<64, FP8>(a, stream);
    case 3: return launch_w<96, FP8>(a, stream);
    case 4: return launch_w<128, FP8>(a, stream);
    case 5: return launch_w<160, FP8>(a, stream);
    case 6: return launch_w<192, FP8>(a, stream);
    case 7: return launch_w<224, FP8>(a, stream);
    case 8: return launch_w<256, FP8>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

size_t kv_attention_ws_bytes(int T, int B, int Hq, int Hkv, int D) {
  const int G = Hq / Hkv;
  if (kv_attention_few_fits(T, B, G)) return kv_attention_few_ws_bytes(Hkv, D);
  const size_t w4 = chunk_division(4).ws_bytes(Hkv, D), w8 = many_rows(T, B, G, D) ? chunk_division(8).ws_bytes(Hkv, D) : 0;
  return w4 > w8 ? w4 : w8;   // (which of the two depends on the page table's columns, too)
}

hipError_t launch_kv_attention(const KvAttnArgs& a, hipStream_t stream) {
  if (kv_attention_few_fits(a.batch.T, a.batch.B, a.G)) return launch_kv_attention_few(a, stream);
  return a.fp8 ? launch_d<true>(a, stream) : launch_d<false>(a, stream);
}

}  // namespace nvfp4moe
