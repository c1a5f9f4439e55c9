// Rotary positions, and the append of new tokens' keys and values to a paged cache (gfx950).
//
// Of each head the dims [start, start + rot) are turned in pairs (u, w), the angle a = position *
// freqs[i] for pair i and a magnitude m:
//   u' = m (u cos a - w sin a)      w' = m (w cos a + u sin a)
// (the transposed rotation, the gradient, with -a). Angles are taken in float64 as turns, whose
// whole part is dropped before they become float32: a position of 10^6 would lose 20 of its 24
// bits otherwise. A workgroup computes the angles of its tokens once, for all their heads. For float32 rows the cosines are
// taken in float64 as well: of a float32 angle, those near 0 have few right bits (outputs off by 3.3e-8, relative,
// instead of 4.9e-8; 1021 tokens of 24 heads 8.5 us either way, 8192 of 8 heads of 128 17.3 instead of 16.9). bf16 and E4M3
// cannot show it.
//
// The append turns the keys (and queries) the same way and writes keys and values where the page
// table puts them, in bf16 or as E4M3(x / scale of the head), rounded once from float32. Values lie
// transposed in their page ([D, page]), as the attention's second product wants them: a workgroup
// takes 64 tokens of one head through LDS, and each store of a wave is of one dim of 64 tokens, 128
// bytes of a page. Tokens that the page table has no page for are left out.
//
// Bound by memory: x is read once and written once. 8192 tokens of 64 heads of 128 in bf16 (268 MB in and out)
// take 51 to 55 us, 4.9 to 5.3 TB/s, what a large copy reaches; a float32 gradient of 25 MB 8.5 us. The append of
// 13 thousand tokens of 64 + 2 x 8 heads of 128 (536 MB) takes 114 to 120 us, 4.5 to 4.7 TB/s: its keys and queries
// alone 104, its transposed values 13; into E4M3 (510 MB) 116, a byte a lane in the values' stores. There the vector units are half busy beside the reads (angles, turns, the
// walk over items), so the walk has no divisions (122 us with them) and angles are computed once for all heads.
// A single token is one dependent chain (sequence, length, page, angles, rows): 3.5 us to turn, 5.2 to append.
#include "common.h"
#include "kernels.h"

namespace nvfp4moe {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 64;      // most tokens of a workgroup
constexpr int kPairs = 4096;     // most angles of a workgroup (32 KB of LDS)
constexpr int kStarts = 1024;    // sequences whose starts fit in LDS

template <int VEC>
__device__ __forceinline__ void load_n(const uint16_t* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else if constexpr (VEC == 4) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(q.x << 16);
    v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16);
    v[3] = __uint_as_float(q.y & 0xffff0000u);
  } else {
    v[0] = bf16_to_f32(*p);
  }
}
template <int VEC>
__device__ __forceinline__ void load_n(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = *p;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + i);
      v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
    }
  }
}
template <int VEC>
__device__ __forceinline__ void store_n(uint16_t* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  else if constexpr (VEC == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
  else
    *p = (uint16_t)f32_to_bf16(v[0]);
}
template <int VEC>
__device__ __forceinline__ void store_n(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    *p = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}
// x / s as it goes to E4M3: saturating at +-448, NaN stays.
__device__ __forceinline__ float to_e4m3_range(float x, float s) {
  const float r = x / s;
  return r != r ? r : fminf(fmaxf(r, -448.0f), 448.0f);
}
template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&v)[VEC], float s) {
  if constexpr (VEC == 1) {
    *p = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(to_e4m3_range(v[0], s), 0.0f, 0, false);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(to_e4m3_range(v[i], s), to_e4m3_range(v[i + 1], s), 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(to_e4m3_range(v[i + 2], s), to_e4m3_range(v[i + 3], s), w, true);
      *reinterpret_cast<int*>(p + i) = w;
    }
  }
}

// cos and sin, times the magnitude, of position * freq; FINE: taken in float64.
template <bool FINE>
__device__ __forceinline__ float2 turn_of(double position, double freq, const RopeTurn& t) {
  const double turns = position * freq * 0.15915494309189533577;   // 1 / (2 pi)
  const double half = 2.0 * (turns - rint(turns));                 // half turns in [-1, 1]
  if constexpr (FINE) {
    double s, c;
    sincospi(half, &s, &c);
    return make_float2((float)(c * t.magnitude), (float)(s * (t.magnitude * t.sign)));
  } else {
    float s, c;
    sincospif((float)half, &s, &c);
    return make_float2(c * t.magnitude, s * (t.magnitude * t.sign));
  }
}

__device__ __forceinline__ double position_at(const void* p, int pos64, int64_t t) {
  return pos64 ? (double)static_cast<const int64_t*>(p)[t] : (double)static_cast<const int*>(p)[t];
}

// A thread's walk over the items of a workgroup's tokens (token, head, item of the head), one of every kThreads:
// divisions at its start alone.
struct Walk {
  int items, heads;   // of a head; of a token
  int dt, dh, dj;     // kThreads items on
};
Walk walk_of(int items, int heads) {
  const int token = items > 0 ? items * heads : 1, rest = kThreads % token;
  return {items, heads, kThreads / token, items > 0 ? rest / items : 0, items > 0 ? rest % items : 0};
}
struct At {
  int t, h, j;
  __device__ __forceinline__ At(const Walk& w) {
    const int i = threadIdx.x, token = w.items * w.heads;
    t = i / token;
    const int r = i - t * token;
    h = r / w.items;
    j = r - h * w.items;
  }
  __device__ __forceinline__ void next(const Walk& w) {
    j += w.dj;
    h += w.dh;
    t += w.dt;
    if (j >= w.items) j -= w.items, ++h;
    if (h >= w.heads) h -= w.heads, ++t;
  }
};

// One item of a head: VEC pairs that are turned, or VEC dims that are not. An item's places in the
// head: the dims [a, a + VEC) and [b, b + VEC).
template <int VEC>
struct Item {
  int a, b, pair;   // pair < 0: dims that are not turned (a alone)
  __device__ __forceinline__ Item(int j, const RopeTurn& t) {
    const int turned = t.rot / (2 * VEC);
    if (j < turned) {
      pair = j * VEC;
      a = t.start + (t.interleaved ? 2 * pair : pair);
      b = a + (t.interleaved ? VEC : t.rot / 2);
    } else {
      a = (j - turned) * VEC;
      a += a < t.start ? 0 : t.rot;
      b = a;
      pair = -1;
    }
  }
};
// One pair (the sums' form is spelt out, so that every width of access rounds alike).
__device__ __forceinline__ void turn_pair(float& u, float& w, const float2 cs) {
  const float x = u, y = w;
  u = __builtin_fmaf(x, cs.x, -(y * cs.y));
  w = __builtin_fmaf(y, cs.x, x * cs.y);
}
template <int VEC>
__device__ __forceinline__ void turn_pairs(float (&u)[VEC], float (&w)[VEC], const float2* cs, bool interleaved) {
  if (interleaved && VEC > 1) {   // u and w hold adjacent pairs: u's first half of the item's pairs, w's the second
#pragma unroll
    for (int i = 0; i + 1 < VEC; i += 2) {
      turn_pair(u[i], u[i + 1], cs[i / 2]);
      turn_pair(w[i], w[i + 1], cs[VEC / 2 + i / 2]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) turn_pair(u[i], w[i], cs[i]);
  }
}

template <typename T, int VEC>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeArgs p, int tokens, Walk walk) {
  extern __shared__ float2 cs[];   // [tokens, rot / 2]
  const int t0 = blockIdx.x * tokens, nt = min(tokens, p.T - t0), half = p.turn.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half;
    cs[i] = turn_of<sizeof(T) == 4>(position_at(p.positions, p.pos64, t0 + t), p.turn.freqs[i - t * half], p.turn);
  }
  __syncthreads();
  const T* x = static_cast<const T*>(p.x.p);
  T* out = static_cast<T*>(const_cast<void*>(p.out.p));
  if (walk.items == 0) return;
  for (At at(walk); at.t < nt; at.next(walk)) {
    const int t = at.t, h = at.h;
    const Item<VEC> it(at.j, p.turn);
    const T* from = x + (t0 + t) * p.x.row + h * p.x.head;
    T* to = out + (t0 + t) * p.out.row + h * p.out.head;
    float u[VEC], w[VEC];
    load_n<VEC>(from + it.a, u);
    if (it.pair >= 0) {
      load_n<VEC>(from + it.b, w);
      turn_pairs<VEC>(u, w, cs + t * half + it.pair, p.turn.interleaved);
      store_n<VEC>(to + it.b, w);
    }
    store_n<VEC>(to + it.a, u);
  }
}

// Where a new token goes.
struct Place {
  double position;     // for its angles
  int64_t page_first;  // first element of its page's heads in the caches (a head holds page * D), or -1: nowhere
  int slot;            // its place in the page
  int row;             // its row, or -1: not a new token
};
__device__ __forceinline__ Place place_of(const KvAppendArgs& p, int t, const int* s_starts) {
  const CacheBatchArgs& b = p.batch;
  Place w = {0.0, -1, 0, -1};
  // the last sequence that starts at t or before (sequences without new tokens start where the next one does)
  const bool in_lds = b.B < kStarts;
  int lo = 0, hi = b.B;   // starts[lo] <= t < starts[hi], if any sequence has row t
  auto start = [&](int i) { return in_lds ? s_starts[i] : b.starts[i]; };
  if (t >= b.T || t < start(0) || t >= start(b.B)) return w;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (start(mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  // (counted from the sequence's last row that is there, as the attention counts)
  const int64_t pos = (int64_t)b.lengths[lo] - min(start(lo + 1), b.T) + t;
  w.row = t;
  w.position = p.positions ? position_at(p.positions, p.pos64, t) : (double)pos;
  const int64_t col = pos >> b.page_log;
  if (pos >= 0 && col < b.cols) {
    const int page = b.page_table[lo * b.ld_table + col];
    if (page >= 0 && page < b.pages) {
      w.page_first = (int64_t)page * p.Hkv * b.page * p.D;
      w.slot = (int)(pos & (b.page - 1));
    }
  }
  return w;
}

// Workgroups [0, turn_groups) turn the queries and keys of `tokens` tokens each; the others take
// the values of v_tokens (a power of two) of one head each, which are not turned.
template <int VEC, bool FP8>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(const KvAppendArgs p, int tokens, int turn_groups,
                                                             int v_tokens_log, Walk walk) {
  extern __shared__ float2 cs[];
  __shared__ Place place[kTokens];
  __shared__ int s_starts[kStarts];
  const CacheBatchArgs& b = p.batch;
  if (b.B < kStarts)
    for (int i = threadIdx.x; i <= b.B; i += kThreads) s_starts[i] = b.starts[i];
  __syncthreads();
  const bool turns = blockIdx.x < (unsigned)turn_groups;
  const int D = p.D;
  if (turns) {
    const int t0 = blockIdx.x * tokens, nt = min(tokens, b.T - t0), half = p.turn.freqs ? p.turn.rot / 2 : 0;
    for (int t = threadIdx.x; t < nt; t += kThreads) place[t] = place_of(p, t0 + t, s_starts);
    __syncthreads();
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int t = i / half;
      cs[i] = turn_of<false>(place[t].position, p.turn.freqs[i - t * half], p.turn);
    }
    __syncthreads();
    for (At at(walk); at.t < nt; at.next(walk)) {
      const int t = at.t;
      int h = at.h;   // key heads, then query heads
      const Item<VEC> it(at.j, p.turn);
      const Place w = place[t];
      const bool key = h < p.Hkv;
      if (w.row < 0 || (key && w.page_first < 0) || (!key && !p.copy && it.pair < 0)) continue;
      if (!key) h -= p.Hkv;
      const HeadRows& rows = key ? p.k : p.q;
      const uint16_t* from = static_cast<const uint16_t*>(rows.p) + w.row * rows.row + h * rows.head;
      float u[VEC], v[VEC];
      load_n<VEC>(from + it.a, u);
      if (it.pair >= 0) {
        load_n<VEC>(from + it.b, v);
        turn_pairs<VEC>(u, v, cs + t * half + it.pair, p.turn.interleaved);
      }
      const int64_t key_at = w.page_first + ((int64_t)h * b.page + w.slot) * D;
      if (key && FP8) {
        uint8_t* to = static_cast<uint8_t*>(p.k_cache) + key_at;
        const float s = p.k_scale ? p.k_scale[h] : 1.0f;
        store_e4m3<VEC>(to + it.a, u, s);
        if (it.pair >= 0) store_e4m3<VEC>(to + it.b, v, s);
      } else {
        uint16_t* to = key ? static_cast<uint16_t*>(p.k_cache) + key_at
                           : static_cast<uint16_t*>(const_cast<void*>(p.q_out.p)) + w.row * p.q_out.row + h * p.q_out.head;
        store_n<VEC>(to + it.a, u);
        if (it.pair >= 0) store_n<VEC>(to + it.b, v);
      }
    }
  } else {
    const int v_tokens = 1 << v_tokens_log, block = blockIdx.x - turn_groups;
    const int h = block % p.Hkv, t0 = (block / p.Hkv) << v_tokens_log, nt = min(v_tokens, b.T - t0);
    uint16_t* tile = reinterpret_cast<uint16_t*>(cs);   // [v_tokens, D + 2]: rows an odd number of words apart
    const int pitch = D + 2;
    for (int t = threadIdx.x; t < v_tokens; t += kThreads)
      place[t] = t < nt ? place_of(p, t0 + t, s_starts) : Place{0.0, -1, 0, -1};
    const uint16_t* from = static_cast<const uint16_t*>(p.v.p) + h * p.v.head;
    if (VEC == 8) {
      for (int i = threadIdx.x; i < nt * (D / 8); i += kThreads) {
        const int t = i / (D / 8), d = (i - t * (D / 8)) * 8;
        const uint4 q = *reinterpret_cast<const uint4*>(from + (t0 + t) * p.v.row + d);
        uint32_t* to = reinterpret_cast<uint32_t*>(tile + t * pitch + d);
        to[0] = q.x, to[1] = q.y, to[2] = q.z, to[3] = q.w;
      }
    } else {
      for (int i = threadIdx.x; i < nt * D; i += kThreads) {
        const int t = i / D, d = i - t * D;
        tile[t * pitch + d] = from[(t0 + t) * p.v.row + d];
      }
    }
    __syncthreads();
    const float s = FP8 && p.v_scale ? p.v_scale[h] : 1.0f;
    // (a thread always has the same token: v_tokens divides kThreads)
    const int t = threadIdx.x & (v_tokens - 1);
    const Place w = place[t];
    if (w.page_first < 0) return;
    const int step = kThreads >> v_tokens_log;
    int64_t at = w.page_first + ((int64_t)h * D + (threadIdx.x >> v_tokens_log)) * b.page + w.slot;
    for (int d = threadIdx.x >> v_tokens_log; d < D; d += step, at += step * b.page) {
      const uint16_t y = tile[t * pitch + d];
      if (FP8)
        static_cast<uint8_t*>(p.v_cache)[at] =
            (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(to_e4m3_range(bf16_to_f32(y), s), 0.0f, 0, false);
      else
        static_cast<uint16_t*>(p.v_cache)[at] = y;
    }
  }
}

// Columns that one access may take: 8, 4 or 1 elements, by the sizes, distances and addresses.
int vector_of(const RopeTurn& t, int D, std::initializer_list<HeadRows> rows, int size) {
  const int rot = t.freqs ? t.rot : 0;
  for (int v = 8; v >= 4; v /= 2) {
    bool fits = rot % (2 * v) == 0 && (rot == 0 || t.start % v == 0) && D % v == 0;
    for (const HeadRows& r : rows)
      fits = fits && (!r.p || (r.row % v == 0 && r.head % v == 0 &&
                               reinterpret_cast<uintptr_t>(r.p) % (size * v < 16 ? size * v : 16) == 0));
    if (fits) return v;
  }
  return 1;
}

// Tokens of a workgroup: about 8192 elements, within its angles' LDS.
int tokens_of(int T, int elements, int half) {
  int n = 8192 / (elements > 0 ? elements : 1);
  n = n < 1 ? 1 : n > kTokens ? kTokens : n;
  if (half > 0 && n * half > kPairs) n = kPairs / half;
  // at least a workgroup for each CU, where there are tokens for them
  const int even = (int)(((int64_t)T + 255) / 256);
  return n < even ? n : even > 0 ? even : 1;
}

// Most workgroups of a launch, which holds fewer than 2^32 threads.
constexpr int64_t kMaxGroups = (int64_t(1) << 32) / kThreads - 1;

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
  const int half = a.turn.rot / 2, tokens = tokens_of(a.T, a.H * a.D, half);
  const int v = vector_of(a.turn, a.D, {a.x, a.out}, a.bf16 ? 2 : 4);
  const int64_t groups = ((int64_t)a.T + tokens - 1) / tokens;
  if (groups > kMaxGroups) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)groups);
  const size_t lds = (size_t)tokens * half * sizeof(float2);
  const Walk walk = walk_of(a.turn.rot / (2 * v) + (a.copy ? (a.D - a.turn.rot) / v : 0), a.H);
  if (a.bf16) {
    auto k = v == 8 ? rope_kernel<uint16_t, 8> : v == 4 ? rope_kernel<uint16_t, 4> : rope_kernel<uint16_t, 1>;
    k<<<grid, kThreads, lds, stream>>>(a, tokens, walk);
  } else {
    auto k = v == 8 ? rope_kernel<float, 8> : v == 4 ? rope_kernel<float, 4> : rope_kernel<float, 1>;
    k<<<grid, kThreads, lds, stream>>>(a, tokens, walk);
  }
  return hipGetLastError();
}

hipError_t launch_kv_append(const KvAppendArgs& a0, hipStream_t stream) {
  KvAppendArgs a = a0;
  if (!a.turn.freqs) a.turn.rot = a.turn.start = 0;
  const int T = a.batch.T, half = a.turn.rot / 2;
  const int tokens = tokens_of(T, (a.Hkv + (a.q.p ? a.Hq : 0)) * a.D, half);
  const int v = vector_of(a.turn, a.D, {a.q, a.q_out, a.k, a.v}, 2);
  int v_log = 0;
  while ((1 << v_log) < kTokens && (1 << v_log) < T) ++v_log;
  const int64_t turn_groups = ((int64_t)T + tokens - 1) / tokens;
  const int64_t groups = turn_groups + (((int64_t)T + (1 << v_log) - 1) >> v_log) * a.Hkv;
  if (groups > kMaxGroups) return hipErrorInvalidConfiguration;
  size_t lds = (size_t)tokens * half * sizeof(float2);
  const size_t v_lds = (size_t)(a.D + 2) * 2 << v_log;
  if (v_lds > lds) lds = v_lds;
  auto k = a.fp8 ? (v == 8 ? kv_append_kernel<8, true> : v == 4 ? kv_append_kernel<4, true> : kv_append_kernel<1, true>)
                 : (v == 8 ? kv_append_kernel<8, false> : v == 4 ? kv_append_kernel<4, false> : kv_append_kernel<1, false>);
  k<<<dim3((unsigned)groups), kThreads, lds, stream>>>(
      a, tokens, (int)turn_groups, v_log, walk_of(half / v + (a.D - 2 * half) / v, a.Hkv + (a.q.p ? a.Hq : 0)));
  return hipGetLastError();
}

}  // namespace nvfp4moe
