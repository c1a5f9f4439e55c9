// Attention of a few new tokens of each sequence over the paged cache (gfx950): the decode step.
//   out[t, h] = sum_j softmax_j(scale q[t, h] . k[j, h / G]) v[j, h / G]   over the keys j that t sees
//
// Bound by the cache's bytes: each visible key and value is read once for the G query heads that
// share it (and for up to 16 / G new tokens): a tile is 16 rows (token, head of the group), the
// width of a matrix instruction. Scores are taken transposed, S^T = K Q^T, so that a lane holds the
// scores of one row; the keys of a block are dealt to the rows of K's operand such that these
// scores are, after the exponential, the operand of the second product O^T = V^T P^T as they lie:
// neither goes through LDS. K and V^T are loaded from the cache straight into operand registers,
// 16 bytes a lane (this is why the cache holds values transposed), two blocks ahead of their use: what a CU has
// under way decides the rate, and registers hold more of it than LDS would.
//
// 64 sequences of 16000 keys, 64 heads over 8 of 128: 719 us in bf16, 5.84 TB/s (plain reads reach 6.0 to 6.5); of
// 500 to 8100 keys 147 us (4.8 TB/s) and 81 us in E4M3 (4.4 TB/s); a sequence of 8000 keys 19 us. What is missing
// there is the start (lengths, page table, first words: 4 us), the last segments' tail and the join (5 to 7 us).
//
// Weights of the second product are two bf16 values each (the rounded exponential, and the rest), so
// that they count as 16 bits; the matrix cores have the time. Running maxima and sums are float32.
//
// The work is divided as Division says; a workgroup of four waves takes one segment, its waves every fourth
// block. Where a tile is split, its parts leave unnormalised sums, which a second launch joins.
#include "gemm_common.h"
#include "kv_attention.h"

namespace nvfp4moe {

namespace {

constexpr int kWaves = kFewWaves;
constexpr int kRows = 16;          // rows of a tile
template <bool FP8>
struct OfCache {
  static constexpr Division kDivision = few_division(FP8);
};

template <int D, bool FP8>
struct Few {
  static constexpr Division kDivision = few_division(FP8);
  static constexpr int kBlockLog = kDivision.block_log, kBlock = 1 << kBlockLog;   // keys of a block
  static constexpr int kTiles = kBlock / 16;       // tiles of 16 keys in the first product
  static constexpr int kDSteps = D / 32;           // its steps
  static constexpr int kPSteps = kBlock / 32;      // steps of the second product
  static constexpr int kDTiles = D / 16;           // its tiles
  // 16-byte words a lane loads of a tile of keys: 32 dims (bf16) or 64 (E4M3, the last one half where
  // 64 does not divide D).
  static constexpr int kKWords = FP8 ? (D + 63) / 64 : D / 32;
};

// WHOLE: a block lies in one page, so that its addresses are the wave's; otherwise each lane looks up its keys' pages.
template <int D, bool FP8, bool WHOLE>
__global__ __launch_bounds__(kWaves* kWave, D > 128 ? 1 : 2) void few_kernel(const KvAttnArgs p) {
  using F = Few<D, FP8>;
  extern __shared__ float lds[];   // [kWaves, 16, D + 4] outputs, then [kWaves, 16, 2] maxima and sums
  const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), c = lane & 15, g = lane >> 4;
  const int h = blockIdx.x % p.Hkv;
  const Segment sg = segment_of<false>(p, F::kDivision, blockIdx.x / p.Hkv);
  if (!sg.found) return;
  const CacheBatchArgs& b = p.batch;

  // This lane's row: new token, query head, and the keys that it sees. (Rows behind the last one see
  // what that one sees, and are not written.)
  const int rows = sg.seq.n * p.G;
  const int row = min(sg.tile * kRows + c, rows - 1), token = row / p.G, head = h * p.G + row - token * p.G;
  const Seen mine = seen_by(sg.seq.position(token), p.window, sg.seq.cap);
  // Keys that every row sees: blocks within need no mask.
  const int first_token = sg.tile * kRows / p.G, last_token = min((sg.tile * kRows + kRows - 1) / p.G, sg.seq.n - 1);
  const int all_lo = seen_by(sg.seq.position(last_token), p.window, sg.seq.cap).lo;
  const int all_hi = seen_by(sg.seq.position(first_token), p.window, sg.seq.cap).hi;

  // This lane's places in a block: for K the key of row c of each tile (rows 4a + i of tile t are key
  // 8a + 4t + i, E4M3 16a + 4t + i), for V and the scores the keys 8g (16g) and on.
  constexpr int kSize = FP8 ? 1 : 2;
  const int page = b.page, page_mask = page - 1;
  const int k_key = (F::kBlock / 4) * (c / 4) + c % 4, v_key = (F::kBlock / 4) * g;
  const int* table = b.page_table + sg.s * b.ld_table;
  const int64_t head_bytes = (int64_t)page * D * kSize;
  struct Pages {
    int k, v;   // of this lane's keys, and values (WHOLE: the same, and the wave's)
  };
  // (columns are checked against the table: a block may end behind it)
  auto pages_of = [&](int block) {
    Pages r = {-1, -1};
    if constexpr (WHOLE) {
      const int col = (block << F::kBlockLog) >> b.page_log;
      if (col < b.cols) r.k = ld_const(table, col);
      r.v = r.k;
    } else {
      // (2 or 4 pages of 16 or 32 keys, in scalar registers)
      const int col = (block << F::kBlockLog) >> b.page_log, k_page = k_key >> b.page_log, v_page = v_key >> b.page_log;
#pragma unroll
      for (int i = 0; i < F::kBlock / 16; ++i) {
        const int at = i < F::kBlock >> b.page_log && col + i < b.cols ? ld_const(table, col + i) : -1;
        r.k = k_page == i ? at : r.k;
        r.v = v_page == i ? at : r.v;
      }
    }
    return r;
  };
  struct Words {
    u32x4v k[F::kTiles][F::kKWords], v[F::kDTiles];
    bool bad;   // this lane's keys have no page
  };
  const uint32_t k_off = (uint32_t)(((WHOLE ? k_key : k_key & page_mask) * D) * kSize + 16 * g);
  const uint32_t v_off = (uint32_t)(((WHOLE ? v_key : v_key & page_mask) + c * page) * kSize);
  const char* k_cache = static_cast<const char*>(p.k_cache) + h * head_bytes;
  const char* v_cache = static_cast<const char*>(p.v_cache) + h * head_bytes;
  auto page_at = [&](int pg) { return (int64_t)(pg >= 0 && pg < b.pages ? pg : 0) * (p.Hkv * head_bytes); };
  auto load_k = [&](int block, const Pages& pg, Words& w) {
    const uint32_t first = (uint32_t)((block << F::kBlockLog) & page_mask) * (D * kSize);   // (not WHOLE: pages start with blocks, or 0)
    const char* at = k_cache + page_at(pg.k);
    const __amdgpu_buffer_rsrc_t r = make_rsrc(at, (uint32_t)head_bytes);
#pragma unroll
    for (int t = 0; t < F::kTiles; ++t)
#pragma unroll
      for (int i = 0; i < F::kKWords; ++i) {
        const uint32_t o = (uint32_t)(4 * t * D * kSize + 64 * i);
        if (!FP8 || 64 * i + 64 <= D) {
          if constexpr (WHOLE)
            w.k[t][i] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(r, k_off + o, first, 0));
          else
            w.k[t][i] = *reinterpret_cast<const u32x4v*>(at + (k_off + first + o));
        } else {   // E4M3, the last 32 dims: 8 bytes a lane
          u32x2 x;
          if constexpr (WHOLE)
            x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, k_off - 8 * g + o, first, 0));
          else
            x = *reinterpret_cast<const u32x2*>(at + (k_off - 8 * g + first + o));
          w.k[t][i] = (u32x4v){x[0], x[1], 0u, 0u};
        }
      }
  };
  auto load_v = [&](int block, const Pages& pg, Words& w) {
    const uint32_t first = (uint32_t)((block << F::kBlockLog) & page_mask) * kSize;
    const char* at = v_cache + page_at(pg.v);
    const __amdgpu_buffer_rsrc_t r = make_rsrc(at, (uint32_t)head_bytes);
    w.bad = pg.v < 0 || pg.v >= b.pages;
#pragma unroll
    for (int d = 0; d < F::kDTiles; ++d) {
      const uint32_t o = (uint32_t)(16 * d * page * kSize);
      if constexpr (WHOLE)
        w.v[d] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(r, v_off, first + o, 0));
      else
        w.v[d] = *reinterpret_cast<const u32x4v*>(at + (v_off + first + o));
    }
  };

  // This wave's blocks: every kWaves-th. Two of them are in registers or on their way: as soon as the keys
  // (values) of one are used up, those of the block two on are requested into their registers.
  const int end = sg.block0 + sg.blocks, block0 = sg.block0 + wave;
  auto ahead = [&](int block) { return min(block, end - 1); };
  Words words[2];
  Pages pages[2];   // of the blocks two and three on
  if (block0 < end) {
    const Pages p0 = pages_of(block0), p1 = pages_of(ahead(block0 + kWaves));
    pages[0] = pages_of(ahead(block0 + 2 * kWaves));
    pages[1] = pages_of(ahead(block0 + 3 * kWaves));
    load_k(block0, p0, words[0]);
    load_v(block0, p0, words[0]);
    if (block0 + kWaves < end) {
      load_k(block0 + kWaves, p1, words[1]);
      load_v(block0 + kWaves, p1, words[1]);
    }
  }
  bf16x8 q[F::kDSteps];
  {
    const uint16_t* at = p.q + (sg.seq.row0 + token) * p.q_row + head * p.q_head;
#pragma unroll
    for (int i = 0; i < F::kDSteps; ++i) {
      // (the order of dims that K's words give)
      const int d = FP8 && i < D / 64 * 2 ? 64 * (i / 2) + 16 * g + 8 * (i % 2) : 32 * i + 8 * g;
      q[i] = *reinterpret_cast<const bf16x8*>(at + d);
    }
  }
  const float log2_scale = p.scale * kLog2e * (FP8 && p.k_scale ? p.k_scale[h] : 1.0f);

  float m = -INFINITY, l = 0.0f;
  f32x4 o[F::kDTiles];
#pragma unroll
  for (int d = 0; d < F::kDTiles; ++d) o[d] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

  auto use = [&](int block, Words& w, Pages& pg) {
    const int then = block + 2 * kWaves;
    const int key0 = (block << F::kBlockLog) + v_key;   // the key of this lane's first score
    f32x4 sc[F::kTiles];
#pragma unroll
    for (int t = 0; t < F::kTiles; ++t) {
      sc[t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < F::kDSteps; ++i) {
        bf16x8 a;
        if constexpr (FP8) {
          const u32x4v x = w.k[t][i / 2];
          a = i % 2 ? e4m3x8_to_bf16(x[2], x[3]) : e4m3x8_to_bf16(x[0], x[1]);
        } else {
          a = __builtin_bit_cast(bf16x8, w.k[t][i]);
        }
        sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, q[i], sc[t], 0, 0, 0);
      }
    }
    if (then < end) load_k(then, pg, w);
    const int begin = block << F::kBlockLog;
    const bool edge = begin < all_lo || begin + F::kBlock > all_hi || __any(w.bad);
    float x[F::kTiles][4], top = -INFINITY;
#pragma unroll
    for (int t = 0; t < F::kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[t][i] = sc[t][i] * log2_scale;
        if (edge) {
          const int key = key0 + 4 * t + i;
          const bool sees = key >= mine.lo && key < mine.hi;
          x[t][i] = !sees ? -INFINITY : w.bad ? NAN : x[t][i];
        }
        top = fmaxf(top, x[t][i]);
      }
    top = max_of_groups(top);
    // (fmaxf leaves NaN out: a row with one gets it from its exponential)
    const float next = fmaxf(m, top), base = next == -INFINITY ? 0.0f : next;
    const float shrink = __builtin_amdgcn_exp2f(m - base);
    m = next;
    float sum = 0.0f;
    bf16x8 hi[F::kPSteps], lo[F::kPSteps];
#pragma unroll
    for (int t = 0; t < F::kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f(x[t][i] - base);
        sum += e;
        const __bf16 r = (__bf16)e;
        hi[t / 2][4 * (t % 2) + i] = r;
        lo[t / 2][4 * (t % 2) + i] = (__bf16)(e - (float)r);
      }
    l = l * shrink + sum;
#pragma unroll
    for (int d = 0; d < F::kDTiles; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[d][i] *= shrink;
    if (edge) {   // values that some row does not see (or no row: what a page holds behind its last token)
#pragma unroll
      for (int d = 0; d < F::kDTiles; ++d) {
#pragma unroll
        for (int u = 0; u < F::kPSteps; ++u) {
          u32x4v bad;
          uint32_t any = 0u;
          u32x4v f;
          if constexpr (FP8)
            f = __builtin_bit_cast(u32x4v, u ? e4m3x8_to_bf16(w.v[d][2], w.v[d][3]) : e4m3x8_to_bf16(w.v[d][0], w.v[d][1]));
          else
            f = w.v[d];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t bits;
            f[i] = finite_bf16x2(f[i], bits);
            bad[i] = bits & 0x3f803f80u;   // 1.0 where one was taken out
            any |= bits;
          }
          if (__any(any != 0u)) {
            // how many of them each row sees; a NaN in the sum where it is any, a zero in their place
            bf16x8 sees;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int key = key0 + 8 * u + i;
              sees[i] = key >= mine.lo && key < mine.hi ? (__bf16)1.0f : (__bf16)0.0f;
            }
            const f32x4 count = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, bad), sees,
                                                                        (f32x4){0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[d][i] = count[i] > 0.0f ? NAN : o[d][i];
            if constexpr (FP8) {   // (E4M3's only ones are its two NaN codes)
              w.v[d][2 * u] = finite_e4m3x4(w.v[d][2 * u]);
              w.v[d][2 * u + 1] = finite_e4m3x4(w.v[d][2 * u + 1]);
            } else {
              w.v[d] = f;
            }
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < F::kPSteps; ++u)
#pragma unroll
      for (int d = 0; d < F::kDTiles; ++d) {
        bf16x8 v;
        if constexpr (FP8)
          v = u ? e4m3x8_to_bf16(w.v[d][2], w.v[d][3]) : e4m3x8_to_bf16(w.v[d][0], w.v[d][1]);
        else
          v = __builtin_bit_cast(bf16x8, w.v[d]);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, hi[u], o[d], 0, 0, 0);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, lo[u], o[d], 0, 0, 0);
      }
    if (then < end) {
      load_v(then, pg, w);
      pg = pages_of(ahead(then + 2 * kWaves));
    }
  };
  for (int block = block0; block < end; block += 2 * kWaves) {
    use(block, words[0], pages[0]);
    if (block + kWaves < end) use(block + kWaves, words[1], pages[1]);
  }
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);

  // Join the waves' sums (this lane: row c, dims 16d + 4g and on).
  constexpr int kPitch = D + 4;
  float* s_ml = lds + kWaves * kRows * kPitch;
  float* s_o = lds + (wave * kRows + c) * kPitch;
#pragma unroll
  for (int d = 0; d < F::kDTiles; ++d) *reinterpret_cast<f32x4*>(s_o + 16 * d + 4 * g) = o[d];
  if (g == 0) {
    s_ml[(wave * kRows + c) * 2] = m;
    s_ml[(wave * kRows + c) * 2 + 1] = l;
  }
  __syncthreads();
  const float v_scale = FP8 && p.v_scale ? p.v_scale[h] : 1.0f;
  for (int i = threadIdx.x; i < min(rows - sg.tile * kRows, kRows) * (D / 8); i += kWaves * kWave) {
    const int r = i / (D / 8), d = (i - r * (D / 8)) * 8;
    float top = -INFINITY, factor[kWaves], total = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_ml[(w * kRows + r) * 2]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      factor[w] = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(s_ml[(w * kRows + r) * 2] - top);
      total += s_ml[(w * kRows + r) * 2 + 1] * factor[w];
    }
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v[j] += lds[(w * kRows + r) * kPitch + d + j] * factor[w];
    }
    if (sg.parts > 1) {
      const Sums part(p, F::kDivision, sg.slot, h);
      *reinterpret_cast<float4*>(part.o + r * D + d) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(part.o + r * D + d + 4) = make_float4(v[4], v[5], v[6], v[7]);
      if (d == 0) {
        part.ml[2 * r] = top;
        part.ml[2 * r + 1] = total;
      }
    } else {
      const int at = sg.tile * kRows + r, t = at / p.G;
      const float f = normalize(sg.seq, t, total, v_scale);
      uint16_t* to = p.out + (sg.seq.row0 + t) * p.o_row + (h * p.G + at - t * p.G) * p.o_head + d;
      *reinterpret_cast<uint4*>(to) = make_uint4(bf16x2(v[0] * f, v[1] * f), bf16x2(v[2] * f, v[3] * f),
                                                 bf16x2(v[4] * f, v[5] * f), bf16x2(v[6] * f, v[7] * f));
    }
  }
}

template <int D, bool FP8, bool WHOLE>
hipError_t launch(const KvAttnArgs& a, hipStream_t stream) {
  using F = Few<D, FP8>;
  const int64_t groups = F::kDivision.segments(a.batch.T, a.batch.B, a.Hkv, a.G) * a.Hkv;
  const size_t lds = (size_t)kWaves * kRows * (D + 4 + 2) * sizeof(float);
  static std::atomic<uint64_t> done{0};
  if (lds > 65536) {
    const hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(few_kernel<D, FP8, WHOLE>), (int)lds, done);
    if (e != hipSuccess) return e;
  }
  few_kernel<D, FP8, WHOLE><<<dim3((unsigned)groups), kWaves * kWave, lds, stream>>>(a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_join<FP8, OfCache<FP8>>(a, stream);
}

template <int D, bool FP8>
hipError_t launch_w(const KvAttnArgs& a, hipStream_t stream) {
  return a.batch.page_log >= Few<D, FP8>::kBlockLog ? launch<D, FP8, true>(a, stream) : launch<D, FP8, false>(a, stream);
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

// Up to 16 rows (token, head of the group) a sequence on average. Tiles of 32 and 64 rows here, one wave a
// SIMD for their sums, were slower than the tiles of 128 rows with most of them empty: 16 sequences of 4
// tokens over 8000 keys (64 heads of 8 groups, D 128, bf16) 155 / 126 us, of 8 tokens 262 / 129 us.
// The host knows the average alone. In batches that mix single tokens (over 200 to 3500 keys each) with one prompt's
// chunk, by tiles of 16 rows / of 128: 32 beside 500 tokens, G 4, E4M3 111 / 77 us, bf16 176 / 81; 63 beside 100, G 8,
// 150 / 92; 95 beside 1400, G 1, which the average sends here, E4M3 232 / 234, but bf16 509 / 266.
bool kv_attention_few_fits(int T, int B, int G) { return (int64_t)T * G <= (int64_t)kRows * B; }

size_t kv_attention_few_ws_bytes(int Hkv, int D) { return few_division(false).ws_bytes(Hkv, D); }

hipError_t launch_kv_attention_few(const KvAttnArgs& a, hipStream_t stream) {
  return a.fp8 ? launch_d<true>(a, stream) : launch_d<false>(a, stream);
}

}  // namespace nvfp4moe
