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
// scales (9/16 or 17/32 byte a weight); the kernels read each of them once and keep as many
// of their loads in flight as registers allow:
//
//   * A wave streams 16-row x 128-column tiles (1 KB of codes in the order of the matrix
//     core's operand, weights_tile.hip) into a register ring D chunks deep, with the lane's
//     scale bytes and its piece of the activations beside them. The columns are dealt out to
//     the waves of a workgroup chunk by chunk, so one 16- or 32-row tile already keeps 8 waves
//     busy and a single token fills the chip; the waves' float32 sums meet in LDS once a tile,
//     in a fixed order.
//   * Persistent workgroups (2 a CU) walk a contiguous range of tiles as one flat sequence of
//     chunks: the ring stays full across tiles and experts.
//   * Activations: the wave itself turns its chunk of the rows into matrix-core operands in a
//     piece of LDS of its own (no barrier). NVFP4 weights are decoded exactly to f16 (E2M1 *
//     E4M3 has at most 6 significant bits), so the rows become f16, scaled by a power of two
//     for each (row, chunk) so that the chunk's largest finite magnitude lies in [2^14, 2^15):
//     exact for bf16 rows down to 2^-31 of that magnitude; the partial product takes the
//     power back when it is added to the float32 sum. MXFP4 weights are decoded exactly to
//     bf16 (whose exponent holds every E8M0 scale), so bf16 rows are used as they are.
//   * The layer's first launch routes in every workgroup (a wave per token; a few microseconds
//     that replace a launch), the second reads the list that workgroup 0 left. An item is an
//     expert with up to 4 of its tokens; an expert with more tokens takes several items.
//   * h between the launches: f16 with a power of two for each 16 columns (NVFP4), bf16 (MXFP4,
//     as its matrix operand needs; the same rounding as h of the W4A16 layer).
//   * The second launch adds a token's experts in its accumulators in ascending expert order: no
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

constexpr int kW = 8;                    // waves per workgroup
constexpr int kNT = kW * kWave;
constexpr int kGrid = 512;               // persistent workgroups: 2 on each of the 256 CUs
constexpr int kRowBytes = 256 + 16;      // LDS bytes of one row's chunk (padded: conflict-free reads)
constexpr int kItemTok = 4;              // tokens of one item of the layer
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
  static __device__ __forceinline__ f32x4 mfma(const Op& a, const Op& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

// Byte offset of the lane's scale bytes of (16-row block blk, chunk c) in the tiled scales.
template <bool MX>
__device__ __forceinline__ uint32_t scale_off(uint32_t blk, uint32_t nch, uint32_t c, uint32_t lane) {
  if (MX) return (blk * ((nch + 15) >> 4) + (c >> 4)) * 1024u + 16u * lane + (c & 15);
  return (blk * ((nch + 7) >> 3) + (c >> 3)) * 1024u + 16u * lane + 2u * (c & 7);
}
template <bool MX>
__device__ __forceinline__ uint32_t ld_scale(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  if (MX) return (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0);
  return ld16(r, off, 0);
}

// Eight bf16 elements of a row's chunk, held by 16 lanes together, as f16 scaled by a power of
// two of the chunk; unscale is the power that takes it back.
__device__ __forceinline__ f16x8 chunk_to_f16(const u32x4& v, float& unscale) {
  u16x2 m = __builtin_bit_cast(u16x2, v[0] & 0x7fff7fffu);
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu));
  uint32_t top = row16_max(max((uint32_t)m[0], (uint32_t)m[1]));
  if (__ballot(top >= 0x7f80u)) {   // an Inf or NaN somewhere: the maximum over the finite ones
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = v[i] & 0x7fffu, hi = (v[i] >> 16) & 0x7fffu;
      t = max(t, lo < 0x7f80u ? lo : 0u);
      t = max(t, hi < 0x7f80u ? hi : 0u);
    }
    top = row16_max(t);
  }
  const uint32_t eb = max(top >> 7, 15u);   // biased exponent of the maximum
  const float scale = __uint_as_float((268u - eb) << 23);
  unscale = __uint_as_float((eb - 14u) << 23);
  f16x8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = (f16)(bf16_to_f32(v[i] & 0xffffu) * scale);
    o[2 * i + 1] = (f16)(__uint_as_float(v[i] & 0xffff0000u) * scale);
  }
  return o;
}

// ------------------------------------------------------------------ matvec, and the layer's first launch
// Waves deal out the chunks ks at a time (ks = 1, 2, 4 or 8: kW / ks groups of waves, each
// with RB row blocks of its own, when K has fewer than 8 chunks).
template <bool MX, bool LAYER, bool SWIGLU, int R, int RB, int D>
__global__ __launch_bounds__(kNT, 4) void few_up_kernel(const FewArgs p) {
  typedef Decode<MX> Dec;
  typedef typename Dec::Op Op;
  static_assert(!SWIGLU || RB == 2, "a gate block and its up block");
  static_assert(!LAYER || (SWIGLU && R == 1), "items of up to 4 tokens");
  constexpr int NTOK = 4 * R;
  constexpr int BUF = R > 1 ? 1 : 2;
  constexpr int REDF = kW * RB * NTOK * 16;
  __shared__ __attribute__((aligned(16))) unsigned char s_row[kW][NTOK * kRowBytes];
  __shared__ float s_unscale[kW][NTOK];
  __shared__ __attribute__((aligned(16))) float s_red[BUF][REDF];
  __shared__ uint32_t s_item[LAYER ? kFewMaxSlots : 1];     // expert << 16 | token mask
  __shared__ uint16_t s_row0[LAYER ? kFewMaxSlots : 1];     // first row of the item in h
  __shared__ uint32_t s_first[LAYER ? kMaxExperts : 1];     // token mask, then item << 16 | row
  __shared__ int s_ids[LAYER ? kFewMaxSlots : 1];
  __shared__ float s_w[LAYER ? kFewMaxSlots : 1];
  __shared__ uint32_t s_n[2];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int T = p.T, K = p.K;
  const uint32_t nch = (uint32_t)(K + kChunk - 1) / kChunk;
  const int KS = 1 << p.ks_log, RG = kW >> p.ks_log;
  const int ksl = wave & (KS - 1), rg = wave >> p.ks_log;
  const int cpw = ((int)nch + KS - 1) >> p.ks_log;       // chunks of a tile for each wave
  const uint32_t nblk = (uint32_t)p.Nw / 16;             // row blocks of a matrix
  const int nsub = SWIGLU ? (int)nblk / 2 : ((int)nblk + RB - 1) / RB;
  const int tpi = (nsub + RG - 1) / RG;                  // tiles of an item
  const uint32_t wbytes = nblk * nch * 1024u;
  const uint32_t sbytes = nblk * (MX ? (nch + 15) >> 4 : (nch + 7) >> 3) * 1024u;
  float fp8_s = 1.0f;

  int nitems = 1;
  if constexpr (LAYER) {
    // ---- routing: a wave per token, then the list of items in ascending expert order
    static_assert(BUF * REDF >= kW * 3 * kWave, "the routing scratch fits");
    const int E = p.E, k = p.k, S = T * k;
    uint32_t* scratch = reinterpret_cast<uint32_t*>(&s_red[0][0]) + wave * 3 * kWave;
    for (int e = tid; e < E; e += kNT) s_first[e] = 0;
    for (int t = wave; t < T; t += kW) {
      const float* row = p.logits + (size_t)t * E;
      if (E <= 256)
        route_token_thresh<4>(row, E, k, lane, s_ids + t * k, s_w + t * k, nullptr, scratch);
      else if (E <= 512)
        route_token_thresh<8>(row, E, k, lane, s_ids + t * k, s_w + t * k, nullptr, scratch);
      else
        route_token_thresh<16>(row, E, k, lane, s_ids + t * k, s_w + t * k, nullptr, scratch);
    }
    float amax = 0.0f;
    if (!MX && p.fp8) {   // one scale for all the rows, from the largest finite magnitude
      const int per = K / 8;
      for (int i = tid; i < T * per; i += kNT) {
        const int t = i / per;
        const uint4 q = *reinterpret_cast<const uint4*>(p.x + (size_t)t * p.ldx + 8 * (i - t * per));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        amax = bf16x8_finite_max(w, amax);
      }
      amax = wave_max(amax);
      if (lane == 0) s_unscale[wave][0] = amax;
    }
    __syncthreads();
    if (!MX && p.fp8) {
      for (int w = 0; w < kW; ++w) amax = fmaxf(amax, s_unscale[w][0]);
      fp8_s = fp8_scale(amax);
    }
    for (int s = tid; s < S; s += kNT) atomicOr(&s_first[s_ids[s]], 1u << (s / k));
    __syncthreads();
    if (wave == 0) {
      const int per = (E + kWave - 1) / kWave;
      uint32_t cnt = 0;   // items << 16 | rows of this lane's experts
      for (int i = 0; i < per; ++i) {
        const int e = lane * per + i;
        const uint32_t n = e < E ? (uint32_t)__popc(s_first[e]) : 0u;
        cnt += ((n + kItemTok - 1) / kItemTok) << 16 | n;
      }
      uint32_t incl = cnt;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const uint32_t up = __shfl_up(incl, o, kWave);
        if (lane >= o) incl += up;
      }
      uint32_t at = incl - cnt;
      for (int i = 0; i < per; ++i) {
        const int e = lane * per + i;
        if (e >= E) break;
        uint32_t m = s_first[e];
        s_first[e] = at;
        while (m) {
          uint32_t part = m;   // the lowest kItemTok tokens of m
#pragma unroll
          for (int j = 0; j < kItemTok; ++j) part &= part - 1;
          part = m & ~part;
          s_item[at >> 16] = (uint32_t)e << 16 | part;
          s_row0[at >> 16] = (uint16_t)(at & 0xffffu);
          at += 0x10000u + (uint32_t)__popc(part);
          m &= ~part;
        }
      }
      if (lane == kWave - 1) s_n[0] = incl >> 16;
    }
    __syncthreads();
    nitems = __builtin_amdgcn_readfirstlane((int)s_n[0]);
    if (blockIdx.x == 0) {   // the list for the second launch
      for (int i = tid; i < nitems; i += kNT) p.plan->item[i] = s_item[i];
      for (int i = tid; i < nitems; i += kNT) p.plan->row0[i] = s_row0[i];
      if (tid == 0) p.plan->n_items = nitems;
      for (int s = tid; s < S; s += kNT) {
        const int t = s / k, e = s_ids[s];
        const uint32_t before = (1u << t) - 1u;
        int rank = 0;   // tokens before t with the same expert
        for (int i = (int)(s_first[e] >> 16); i < nitems && (int)(s_item[i] >> 16) == e; ++i)
          rank += __popc(s_item[i] & before);
        p.plan->weight[(s_first[e] & 0xffffu) + rank] = MX ? s_w[s] : s_w[s] * p.g_down[e];
      }
    }
  }

  // ---- this workgroup's tiles, as one flat sequence of chunks
  const int64_t ntiles = (int64_t)nitems * tpi;
  const int t0 = (int)(ntiles * blockIdx.x / gridDim.x);
  const int t1 = (int)(ntiles * (blockIdx.x + 1) / gridDim.x);
  if (t0 >= t1) return;
  const int nst = (t1 - t0) * cpw;

  const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x, (uint32_t)((p.ldx * (T - 1) + K) * 2));
  __amdgpu_buffer_rsrc_t wr, sr;
  uint32_t xoff[R];
  auto item_word = [&](int it) -> uint32_t {
    return LAYER ? (uint32_t)__builtin_amdgcn_readfirstlane((int)s_item[it]) : (1u << T) - 1u;
  };
  auto open_item = [&](int it) {   // the loads' side of an item: its matrix and its token rows
    const uint32_t w = item_word(it);
    const size_t e = LAYER ? w >> 16 : 0;
    wr = make_rsrc(p.codes + e * wbytes, wbytes);
    sr = make_rsrc(p.scales + e * sbytes, sbytes);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      int tok = -1;
      if (LAYER) {
        uint32_t m = w & 0xffffu;
        for (int q = 0; m; ++q, m &= m - 1) tok = q == g ? __builtin_ctz(m) : tok;
      } else {
        tok = 4 * r + g < T ? 4 * r + g : -1;
      }
      xoff[r] = tok >= 0 ? (uint32_t)(tok * p.ldx * 2) + 16u * l16 : kOOB;
    }
  };

  u32x4 wring[D][RB], xring[D][R];
  uint32_t sring[D][RB];
  int it_l = t0 / tpi, tile_l = t0 - it_l * tpi, step_l = 0, left_l = nst;   // the loads' position
  open_item(it_l);
  auto issue = [&](int d) {
    const uint32_t c = (uint32_t)(ksl + (step_l << p.ks_log));
    const uint32_t sub = (uint32_t)(tile_l * RG + rg);
    const bool ok = left_l > 0 && c < nch && sub < (uint32_t)nsub;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const uint32_t blk = SWIGLU ? sub + (b ? nblk / 2 : 0) : sub * RB + b;
      const bool in = ok && blk < nblk;
      wring[d][b] = ld128(wr, in ? 16u * lane + (blk * nch + c) * 1024u : kOOB, 0);
      sring[d][b] = ld_scale<MX>(sr, in ? scale_off<MX>(blk, nch, c, lane) : kOOB);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      xring[d][r] = ld128(xr, ok && (int)(c * kChunk) + 8 * l16 < K && xoff[r] != kOOB ? xoff[r] + c * 256u : kOOB, 0);
    --left_l;
    if (++step_l == cpw) {
      step_l = 0;
      if (++tile_l == tpi) {
        tile_l = 0;
        if (left_l > 0) open_item(++it_l);
      }
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) issue(d);

  int it = t0 / tpi, tile = t0 - it * tpi, step = 0, done = 0, buf = 0;
  f32x4 tot[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) tot[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
  unsigned char* row = s_row[wave];
  const int ntok = LAYER ? NTOK : T;

  for (int s = 0; s < nst; s += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (s + d < nst) {
        const uint32_t c = (uint32_t)(ksl + (step << p.ks_log));
        const int sub = tile * RG + rg;
        if (c < nch && sub < nsub) {
          // the rows' chunk into the wave's LDS
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (R == 1 || 4 * r < T) {
              u32x4 v = xring[d][r];
              if (MX) {
                *reinterpret_cast<u32x4*>(row + (4 * r + g) * kRowBytes + 16 * l16) = v;
              } else {
                if (LAYER && p.fp8) {
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    v[i] = fp8_roundtrip_bits(bf16_to_f32(v[i] & 0xffffu), fp8_s) |
                           fp8_roundtrip_bits(__uint_as_float(v[i] & 0xffff0000u), fp8_s) << 16;
                }
                float un;
                const f16x8 h = chunk_to_f16(v, un);
                *reinterpret_cast<f16x8*>(row + (4 * r + g) * kRowBytes + 16 * l16) = h;
                if (l16 == 0) s_unscale[wave][4 * r + g] = un;
              }
            }
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          const int fr = l16 & (NTOK - 1);
          Op bf[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            bf[j] = *reinterpret_cast<const Op*>(row + fr * kRowBytes + 64 * g + 16 * j);
          const float un = MX ? 1.0f : s_unscale[wave][fr];
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            Op wf[4];
            Dec::run(wring[d][b], sring[d][b], wf);
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
        }
        if (++step == cpw) {
          // ---- a tile is complete: the waves' sums, then the epilogue
          step = 0;
          float* red = s_red[buf];
          if (l16 < NTOK) {
#pragma unroll
            for (int b = 0; b < RB; ++b)
              *reinterpret_cast<f32x4*>(&red[((wave * RB + b) * NTOK + l16) * 16 + 4 * g]) = tot[b];
          }
#pragma unroll
          for (int b = 0; b < RB; ++b) tot[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
          __syncthreads();
          const uint32_t iw = item_word(it);
          const int n = LAYER ? __popc(iw & 0xffffu) : ntok;
          const float alpha = MX ? 1.0f : ld_const(p.g, LAYER ? iw >> 16 : 0);
          constexpr int NB = SWIGLU ? 1 : RB;
          const int total = RG * NB * n * 16;
          // a different wave starts each tile, so that short epilogues spread over the SIMDs
          for (int i = (tid + kWave * done) & (kNT - 1); i < total; i += kNT) {
            const int r16 = i & 15, q = i >> 4;
            const int grp = q / (NB * n), b = (q / n) % NB, col = q % n;
            const int osub = tile * RG + grp;
            float v = 0.0f, u = 0.0f;
            for (int w = 0; w < KS; ++w) {
              const float* a = &red[(((grp * KS + w) * RB + b) * NTOK + col) * 16 + r16];
              v += a[0];
              if (SWIGLU) u += a[NTOK * 16];
            }
            v *= alpha;
            if (SWIGLU) v = swiglu1(v, u * alpha);
            if constexpr (LAYER) {
              const uint32_t hr = (uint32_t)s_row0[it] + (uint32_t)col;
              const int F = p.Nw / 2, f = osub * 16 + r16;
              if (MX) {
                if (osub < nsub) static_cast<uint16_t*>(p.h)[(size_t)hr * F + f] = (uint16_t)f32_to_bf16(v);
              } else {
                const uint32_t top = row16_max(finite_abs_bits(v));
                const int e2 = top ? max((int)(top >> 23) - 141, kNoExp) : kNoExp;
                if (osub < nsub) {
                  static_cast<f16*>(p.h)[(size_t)hr * F + f] = (f16)ldexpf(v, -e2);
                  if (r16 == 0) p.hexp[(size_t)hr * (F / 16) + osub] = (int8_t)e2;
                }
              }
            } else {
              const uint32_t blk = SWIGLU ? (uint32_t)osub : (uint32_t)(osub * RB + b);
              if (osub < nsub && blk < (SWIGLU ? nblk / 2 : nblk)) {
                const size_t n0 = (size_t)blk * 16 + r16;
                if (p.add) {
                  const size_t ao = (size_t)col * p.ld_add + n0;
                  v += p.add_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.add)[ao])
                                  : static_cast<const float*>(p.add)[ao];
                }
                const size_t o = (size_t)col * p.ld_out + n0;
                if (p.out_bf16)
                  static_cast<uint16_t*>(p.out)[o] = (uint16_t)f32_to_bf16(v);
                else
                  static_cast<float*>(p.out)[o] = v;
              }
            }
          }
          if (BUF == 1) __syncthreads();
          else buf ^= 1;
          ++done;
          if (++tile == tpi) {
            tile = 0;
            ++it;
          }
        }
      }
      issue(d);
    }
  }
}

// ------------------------------------------------------------------ the layer's second launch
// One workgroup per RB blocks of 16 output columns; its waves deal out the (item, chunk) pairs.
template <bool MX, int RB, int D>
__global__ __launch_bounds__(kNT, 4) void few_down_kernel(const FewArgs p) {
  typedef Decode<MX> Dec;
  typedef typename Dec::Op Op;
  __shared__ __attribute__((aligned(16))) unsigned char s_row[kW][kItemTok * kRowBytes];
  __shared__ float s_mul[kW][kItemTok];
  __shared__ __attribute__((aligned(16))) float s_red[kW * RB][16 * 16];
  __shared__ uint32_t s_item[kFewMaxSlots];
  __shared__ uint16_t s_row0[kFewMaxSlots];
  __shared__ float s_w[kFewMaxSlots];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int T = p.T, F = p.K, S = T * p.k;
  const uint32_t nch = (uint32_t)(F + kChunk - 1) / kChunk;
  const uint32_t nblk = (uint32_t)p.Nw / 16;
  const uint32_t wbytes = nblk * nch * 1024u;
  const uint32_t sbytes = nblk * (MX ? (nch + 15) >> 4 : (nch + 7) >> 3) * 1024u;

  const int nitems = __builtin_amdgcn_readfirstlane(p.plan->n_items);
  for (int i = tid; i < nitems; i += kNT) s_item[i] = p.plan->item[i];
  for (int i = tid; i < nitems; i += kNT) s_row0[i] = p.plan->row0[i];
  for (int i = tid; i < S; i += kNT) s_w[i] = p.plan->weight[i];
  __syncthreads();

  const int npair = nitems * (int)nch;
  const int nst = wave < npair ? (npair - wave + kW - 1) / kW : 0;   // this wave's pairs
  const __amdgpu_buffer_rsrc_t hr = make_rsrc(p.h, (uint32_t)S * (uint32_t)F * 2u);
  const __amdgpu_buffer_rsrc_t er = make_rsrc(p.hexp, (uint32_t)S * (uint32_t)(F / 16));
  __amdgpu_buffer_rsrc_t wr, sr;
  uint32_t hrow = 0;   // row of h for this lane's 16-lane group (kOOB: none)
  auto open_item = [&](int a) {
    const uint32_t w = (uint32_t)__builtin_amdgcn_readfirstlane((int)s_item[a]);
    wr = make_rsrc(p.codes + (size_t)(w >> 16) * wbytes, wbytes);
    sr = make_rsrc(p.scales + (size_t)(w >> 16) * sbytes, sbytes);
    hrow = g < __popc(w & 0xffffu) ? (uint32_t)s_row0[a] + (uint32_t)g : kOOB;
  };
  u32x4 wring[D][RB], xring[D];
  uint32_t sring[D][RB];
  int ering[D];
  int a_l = wave / (int)nch, c_l = wave - a_l * (int)nch, left_l = nst;
  if (nst > 0) open_item(a_l);
  auto issue = [&](int d) {
    const bool ok = left_l > 0;
    const uint32_t c = (uint32_t)c_l;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const uint32_t blk = blockIdx.x * RB + b;
      const bool in = ok && blk < nblk;
      wring[d][b] = ld128(wr, in ? 16u * lane + (blk * nch + c) * 1024u : kOOB, 0);
      sring[d][b] = ld_scale<MX>(sr, in ? scale_off<MX>(blk, nch, c, lane) : kOOB);
    }
    const bool in = ok && hrow != kOOB && (int)(c * kChunk) + 8 * l16 < F;
    xring[d] = ld128(hr, in ? (hrow * (uint32_t)F + c * kChunk + 8u * l16) * 2u : kOOB, 0);
    if (!MX) ering[d] = (int)(int8_t)__builtin_amdgcn_raw_buffer_load_b8(er, in ? hrow * (uint32_t)(F / 16) + c * 8u + l16 / 2u : kOOB, 0, 0);
    --left_l;
    c_l += kW;
    if (c_l >= (int)nch) {
      do {
        c_l -= (int)nch;
        ++a_l;
      } while (c_l >= (int)nch);
      if (left_l > 0) open_item(a_l);
    }
  };
  if (nst > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) issue(d);
  }

  f32x4 tot[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) tot[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
  int a = wave / (int)nch, c = wave - a * (int)nch;
  bool has = false;     // the lane's token is one of the item's
  int fr = 0;           // and its place among them
  float mul = 0.0f;     // the weight (times the global scale) of the row of this lane's group
  auto take_item = [&](int i) {
    const uint32_t w = (uint32_t)__builtin_amdgcn_readfirstlane((int)s_item[i]);
    has = (w >> l16) & 1u;
    fr = __popc(w & ((1u << l16) - 1u)) & (kItemTok - 1);
    mul = g < __popc(w & 0xffffu) ? s_w[s_row0[i] + g] : 0.0f;
  };
  if (nst > 0) take_item(a);
  unsigned char* row = s_row[wave];
  for (int s = 0; s < nst; s += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (s + d < nst) {
        if (MX) {
          *reinterpret_cast<u32x4*>(row + g * kRowBytes + 16 * l16) = xring[d];
          if (l16 == 0) s_mul[wave][g] = mul;
        } else {
          // the chunk's blocks of 16 columns to one power of two
          const int e2 = c * kChunk + 8 * l16 < F ? ering[d] : kNoExp;
          const int top = (int)row16_max((uint32_t)(e2 + 256)) - 256;
          const f16 f = (f16)ldexpf(1.0f, e2 - top);
          const f16x8 v = __builtin_bit_cast(f16x8, xring[d]) * f;
          *reinterpret_cast<f16x8*>(row + g * kRowBytes + 16 * l16) = v;
          if (l16 == 0) s_mul[wave][g] = ldexpf(mul, top);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        Op bf[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) bf[j] = *reinterpret_cast<const Op*>(row + fr * kRowBytes + 64 * g + 16 * j);
        const float m = s_mul[wave][fr];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          Op wf[4];
          Dec::run(wring[d][b], sring[d][b], wf);
          f32x4 acc = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 4; ++j) acc = Dec::mfma(wf[j], bf[j], acc);
          // only the item's own tokens: the other columns hold products that mean nothing
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[b][i] = has ? fmaf(acc[i], m, tot[b][i]) : tot[b][i];
        }
        c += kW;
        if (c >= (int)nch) {
          do {
            c -= (int)nch;
            ++a;
          } while (c >= (int)nch);
          if (s + d + 1 < nst) take_item(a);
        }
      }
      issue(d);
    }
  }

#pragma unroll
  for (int b = 0; b < RB; ++b) *reinterpret_cast<f32x4*>(&s_red[wave * RB + b][l16 * 16 + 4 * g]) = tot[b];
  __syncthreads();
  for (int i = tid; i < RB * T * 16; i += kNT) {
    const int r16 = i & 15, q = i >> 4, b = q / T, t = q - b * T;
    const uint32_t blk = blockIdx.x * RB + b;
    if (blk >= nblk) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kW; ++w) v += s_red[w * RB + b][t * 16 + r16];
    static_cast<uint16_t*>(p.out)[(size_t)t * p.ld_out + blk * 16 + r16] = (uint16_t)f32_to_bf16(v);
  }
}

// Groups of chunks a wave of the workgroup takes its turn in: 8 when every wave then has a chunk.
int ks_log_for(int K) {
  const int nch = (K + kChunk - 1) / kChunk;
  return nch >= 8 ? 3 : nch >= 4 ? 2 : nch >= 2 ? 1 : 0;
}

template <bool MX, bool SWIGLU, int R, int RB, int D>
hipError_t launch_mv(const FewArgs& a, hipStream_t stream) {
  const int nblk = a.Nw / 16, rg = kW >> a.ks_log;
  const int nsub = SWIGLU ? nblk / 2 : (nblk + RB - 1) / RB;
  const int tiles = (nsub + rg - 1) / rg;
  few_up_kernel<MX, false, SWIGLU, R, RB, D><<<tiles < kGrid ? tiles : kGrid, kNT, 0, stream>>>(a);
  return hipGetLastError();
}

template <bool MX, bool SWIGLU>
hipError_t launch_mv_rows(const FewArgs& a, hipStream_t stream) {
  if (a.T <= 4) return launch_mv<MX, SWIGLU, 1, 2, 4>(a, stream);
  return launch_mv<MX, SWIGLU, 4, 2, 2>(a, stream);
}

}  // namespace

hipError_t launch_few_matvec(FewArgs a, bool mx, bool swiglu, hipStream_t stream) {
  a.ks_log = ks_log_for(a.K);
  if (mx) return swiglu ? launch_mv_rows<true, true>(a, stream) : launch_mv_rows<true, false>(a, stream);
  return swiglu ? launch_mv_rows<false, true>(a, stream) : launch_mv_rows<false, false>(a, stream);
}

hipError_t launch_few_layer(FewArgs up, FewArgs down, bool mx, hipStream_t stream) {
  up.ks_log = ks_log_for(up.K);
  const int rg = kW >> up.ks_log, nsub = up.Nw / 32;
  const int64_t tiles = (int64_t)up.T * up.k * ((nsub + rg - 1) / rg);   // bound: every slot an item
  const int grid = tiles < kGrid ? (int)tiles : kGrid;
  if (mx)
    few_up_kernel<true, true, true, 1, 2, 4><<<grid, kNT, 0, stream>>>(up);
  else
    few_up_kernel<false, true, true, 1, 2, 4><<<grid, kNT, 0, stream>>>(up);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int RB = 1;
  const int wgs = (down.Nw / 16 + RB - 1) / RB;
  if (mx)
    few_down_kernel<true, RB, 4><<<wgs, kNT, 0, stream>>>(down);
  else
    few_down_kernel<false, RB, 4><<<wgs, kNT, 0, stream>>>(down);
  return hipGetLastError();
}

}  // namespace nvfp4moe
