// Top-k of one token by one wave: shared by the routers (route.hip) and the few-token layer
// (few_rows.hip), so that both keep the same experts in the same order with the same weights.
#pragma once

#include "common.h"

namespace nvfp4moe {

// Order-preserving uint32 key of a logit (NaN as -inf, -0 as +0): key order = value order.
__device__ __forceinline__ uint32_t logit_key(float x) {
  if (x != x) x = -INFINITY;
  if (x == 0.0f) x = 0.0f;
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int wave_count(bool pred) { return __popcll(__ballot(pred)); }

// Top-k of one token by one wave, in k rounds of wave argmax: each round takes the largest
// order-preserving logit key (DPP max over the wave) and, among the experts holding it, the lowest
// id (ballots; registers ascend in id, lanes within a register), and removes it. Lane r holds rank
// r. w: the kept experts' softmax, in double and rounded once; without SOFTMAX their logits.
template <int PL, bool SOFTMAX = true>
__device__ __forceinline__ void route_token_rounds(const float* __restrict__ row, int E, int k, int lane,
                                                   int* __restrict__ ids, float* __restrict__ w, int* lds_ids) {
  uint32_t key[PL];
  float v[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + kWave * i;
    const float x = e < E ? row[e] : -INFINITY;
    v[i] = (x != x) ? -INFINITY : x;
    key[i] = e < E ? logit_key(x) : 0u;   // every real key is >= logit_key(-inf) > 0
  }
  int my_e = 0;
  float my_x = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < PL; ++i) best = max(best, key[i]);
    best = wave_max_u32_uniform(best);
    int e = -1;
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const uint64_t m = __ballot(key[i] == best);
      if (e < 0 && m) {
        const int l = __builtin_ctzll(m);
        e = kWave * i + l;
        x = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v[i]), l));
      }
    }
    if (lane == j) {
      my_e = e;
      my_x = x;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (kWave * i + lane == e) key[i] = 0u;
  }
  if (!SOFTMAX) {
    if (lane < k) {
      ids[lane] = my_e;
      w[lane] = my_x;
    }
    return;
  }
  const double m = (double)__uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(my_x), 0));
  const double ex = lane < k ? exp((double)my_x - m) : 0.0;
  double sum = ex;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  if (lane < k) {
    ids[lane] = my_e;
    w[lane] = (float)(ex / sum);
    lds_ids[lane] = my_e;
  }
}

// The same without k serial rounds (same ids, order and weights; its cost does not grow with k):
// the k-th largest key th is found bit by bit (the largest th with at least k keys >= th; a
// ballot per register and bit), the keys above th are kept and the lowest ids among those
// equal to th fill the rest, the k kept (key, id, logit) go to the wave's LDS scratch in id
// order, lane j takes entry j and counts the kept entries ahead of it (larger key, or equal
// key and lower id), and lane r then takes the entry of rank r, as round r would have.
// scratch: 3 x 64 words of the wave's own LDS. w: the kept experts' softmax, in double and rounded
// once; without SOFTMAX their logits, largest first.
template <int PL, bool SOFTMAX = true>
__device__ __forceinline__ void route_token_thresh(const float* __restrict__ row, int E, int k, int lane,
                                                   int* __restrict__ ids, float* __restrict__ w, int* lds_ids,
                                                   uint32_t* scratch) {
  uint32_t key[PL];
  float v[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + kWave * i;
    const float x = e < E ? row[e] : -INFINITY;
    v[i] = (x != x) ? -INFINITY : x;
    key[i] = e < E ? logit_key(x) : 0u;   // every real key is >= logit_key(-inf) > 0
  }
  uint32_t th = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = th | (1u << bit);
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) cnt += wave_count(key[i] >= cand);
    if (cnt >= k) th = cand;
    if (cnt == k) break;   // exactly the kept ones lie at or above th
  }
  int need = k;
#pragma unroll
  for (int i = 0; i < PL; ++i) need -= wave_count(key[i] > th);
  const uint64_t below = lane == 0 ? 0ull : (~0ull >> (64 - lane));
  int base = 0;   // kept entries in the registers before i (ids ascend with i, then lane)
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const uint64_t eq = __ballot(key[i] == th);
    const bool kept = key[i] > th || (((eq >> lane) & 1ull) && __popcll(eq & below) < need);
    const int c = __popcll(eq);
    need = need > c ? need - c : 0;
    const uint64_t km = __ballot(kept);
    if (kept) {
      const int pos = base + __popcll(km & below);
      scratch[pos] = key[i];
      scratch[kWave + pos] = (uint32_t)(lane + kWave * i);
      scratch[2 * kWave + pos] = __float_as_uint(v[i]);
    }
    base += __popcll(km);
  }
  uint32_t kj = 0, ej = 0, xj = 0;
  if (lane < k) {
    kj = scratch[lane];
    ej = scratch[kWave + lane];
    xj = scratch[2 * kWave + lane];
  }
  int rank = 0;
  for (int m = 0; m < k; ++m) {
    const uint32_t km = (uint32_t)__builtin_amdgcn_readlane((int)kj, m);
    const uint32_t em = (uint32_t)__builtin_amdgcn_readlane((int)ej, m);
    rank += (km > kj || (km == kj && em < ej)) ? 1 : 0;
  }
  if (lane < k) {
    scratch[rank] = ej;
    scratch[kWave + rank] = xj;
  }
  int my_e = 0;
  float my_x = 0.0f;
  if (lane < k) {
    my_e = (int)scratch[lane];
    my_x = __uint_as_float(scratch[kWave + lane]);
  }
  if (!SOFTMAX) {
    if (lane < k) {
      ids[lane] = my_e;
      w[lane] = my_x;
    }
    return;
  }
  const double m = (double)__uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(my_x), 0));
  const double ex = lane < k ? exp((double)my_x - m) : 0.0;
  double sum = ex;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  if (lane < k) {
    ids[lane] = my_e;
    w[lane] = (float)(ex / sum);
    if (lds_ids) lds_ids[lane] = my_e;
  }
}

}  // namespace nvfp4moe
