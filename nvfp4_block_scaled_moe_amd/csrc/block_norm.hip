// The norms around a block with its gate and residual scale (gfx950), in one pass over the rows:
//   u    = y                                      y / sqrt(mean(y^2) + eps) * (o + post_w)  with post_w
//   r'   = r + scale * gate * u
//   next = bf16( r' / sqrt(mean(r'^2) + eps) * (o + pre_w) )                               with pre_w
// y is the block's output, or the experts' rows with their weights: y_t = sum_j w[t, j] Y[row of
// slot (t, j)] in ascending j (the unpermute-reduce, whose bf16 output then never exists); y_add
// (a shared expert's output) is added to either. Without y only next is written (the norm before
// the first block).
//
// Memory-bound: y (k rows of it for the experts' form), r and a full gate are read once, r' and
// next written once; everything between stays in registers. One workgroup a row: a thread holds
// V groups of 8 consecutive columns (16- and 32-byte accesses), the two sums of squares meet in
// LDS (float32: at most 32 squares a thread, then a tree over lanes and waves). Next is computed
// from r' in float32, before r' is rounded to its stored type.
//
// 8192 rows of 7168 (y and next bf16, r float32: 704 MB): 144 us, 4.9 TB/s, where a copy reaches
// 5.1-5.2; with one group a thread 165 us, with the weights requested ahead, too, 167 (fewer
// workgroups a CU), with r requested behind y 152. The experts' rows (float32, 8 a token, 6144 columns,
// bf16 r): 4096 tokens (957 MB) 194 us, 4.9 TB/s; 1024 57 us and 256 15.0 us, 0.8 of the copy rate.
// One row of 8 x 6144: 6.2 us, of 37 x 1000: 3.0 us, bound by the latency of the launch and of
// two dependent reads; requested one after the other, as they are used, the tensors took 1.0 and 0.7
// us more.
#include "gemm_common.h"
#include "kernels.h"

namespace nvfp4moe {

namespace {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormManyRows = 256; // rows from which a thread holds more columns

// Eight consecutive values of a row as they lie in memory: 16 bytes of bf16, or 32 of float32.
// The loads of both types are the same two (the second out of range for bf16, and both past the
// row's end: such loads return zeros and touch no memory), so that they can all be requested
// before the first is waited for; a branch on the type would wait in each of its sides.
struct Raw8 {
  u32x4 a, b;
};
struct Row {   // a row of H values of one tensor; bytes 0: absent, reads as zeros
  __amdgpu_buffer_rsrc_t r;
  bool bf16;
  __device__ __forceinline__ Row(const void* p, bool is_bf16, int64_t first, int H)
      : r(make_rsrc(static_cast<const char*>(p) + first * (is_bf16 ? 2 : 4), p ? (uint32_t)H * (is_bf16 ? 2u : 4u) : 0u)),
        bf16(is_bf16) {}
  __device__ __forceinline__ Raw8 load(int col) const {
    const uint32_t o = (uint32_t)col * (bf16 ? 2u : 4u);
    return {ld128(r, o, 0), ld128(r, bf16 ? kOOB : o + 16u, 0)};
  }
  __device__ __forceinline__ void values(const Raw8& q, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(bf16 ? q.a[i] << 16 : i < 2 ? q.a[2 * i] : q.b[2 * i - 4]);
      v[2 * i + 1] = __uint_as_float(bf16 ? q.a[i] & 0xffff0000u : i < 2 ? q.a[2 * i + 1] : q.b[2 * i - 3]);
    }
  }
};

__device__ __forceinline__ void store8(void* p, bool bf16, int64_t o, const float (&v)[8]) {
  if (bf16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + o) =
        make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  } else {
    float* q = static_cast<float*>(p) + o;
    *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// One step of a sum over lanes by DPP moves: 0-3 leave a row of 16's sum in all its lanes, 4 and 5
// fold the four rows into lane 63.
template <int S>
__device__ __forceinline__ float dpp_add(float v) {
  constexpr int ctrl[6] = {0xb1, 0x4e, 0x141, 0x140, 0x142, 0x143};
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl[S], S == 4 ? 0xa : S == 5 ? 0xc : 0xf,
                                                        0xf, false));
}
__device__ __forceinline__ float row16_sum(float v) { return dpp_add<3>(dpp_add<2>(dpp_add<1>(dpp_add<0>(v)))); }

// Sum over the workgroup of nw waves, in every thread; part: kNormMaxThreads / 64 floats of LDS of its own.
__device__ __forceinline__ float block_sum(float v, float* part, int nw) {
  v = dpp_add<5>(dpp_add<4>(row16_sum(v)));
  v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
  if (nw == 1) return v;
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  const int l = threadIdx.x & 15;
  return row16_sum(l < nw ? part[l] : 0.0f);
}

template <int V, bool ROWS>
__global__ __launch_bounds__(kNormMaxThreads) void block_norm_kernel(const BlockNormArgs p) {
  // The arguments, one of each 64 bytes of them, requested together (each misses every cache).
  static_assert(sizeof(BlockNormArgs) <= 256, "four lines");
  asm volatile("" ::"s"(p.r_bf16), "s"(p.k), "s"(p.gate_bf16), "s"(p.nt));
  static_assert(kNormMaxThreads / kWave <= 16, "a row of lanes holds the waves' sums");
  // One group of columns a thread (short rows, where latency counts): everything is requested
  // before anything is waited for. More groups: registers allow less.
  constexpr bool kAll = V == 1, kResid = !(ROWS && V == 4);
  constexpr int kBatch = V == 4 ? 2 : 4;   // experts' rows requested together
  __shared__ float part[2][kNormMaxThreads / kWave];
  const int64_t t = blockIdx.x;
  const int H = p.H, nw = p.nt / kWave;
  int col[V];
#pragma unroll
  for (int v = 0; v < V; ++v) col[v] = ((int)threadIdx.x + v * p.nt) * 8;

  // The experts' rows: a lane for each of the token's slots, its row and weight. (Requested first:
  // loads return in order.)
  static_assert(kMaxTopK <= kWave, "a lane for each slot");
  const int lane = threadIdx.x % kWave;
  int row_of = 0;
  float slot_w = 0.0f;
  if (ROWS) {
    const int64_t slot = t * p.k + min(lane, p.k - 1);
    row_of = p.slot_to_row[slot];
    slot_w = p.topk_w[slot];
  }
  const Row resid(p.resid, p.r_bf16, t * p.ld_r, H), y_add(p.y_add, p.ya_bf16, t * p.ld_ya, H);
  const Row post_w(p.post_w, p.w_bf16, 0, H), pre_w(p.pre_w, p.w_bf16, 0, H);
  const Row gate(p.gate_col ? p.gate : nullptr, p.gate_bf16, t * p.gate_row, H);
  Raw8 rq[V], aq[V], gq[V], oq[V], nq[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (kResid) rq[v] = resid.load(col[v]);
    if (kAll) {
      aq[v] = y_add.load(col[v]);
      oq[v] = post_w.load(col[v]);
      gq[v] = gate.load(col[v]);
      nq[v] = pre_w.load(col[v]);
    }
  }
  float r[V][8], y[V][8];
  if (ROWS) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[v][i] = 0.0f;
    const int weight_of = __float_as_int(lane < p.k ? slot_w : 0.0f);   // (with a row of zeros: adds nothing)
    for (int j0 = 0; j0 < p.k; j0 += kBatch) {
      int row[kBatch];
      float w[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int l = min(j0 + j, kWave - 1);
        row[j] = __builtin_amdgcn_readlane(row_of, l);
        w[j] = __int_as_float(__builtin_amdgcn_readlane(weight_of, l));
      }
      const Row first(p.y, p.y_bf16, 0, H);
      Raw8 q[kBatch][V];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const Row yr(j0 + j < p.k ? p.y : nullptr, p.y_bf16, row[j] * p.ld_y, H);
#pragma unroll
        for (int v = 0; v < V; ++v) q[j][v] = yr.load(col[v]);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float u[8];
          first.values(q[j][v], u);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[v][i] = fmaf(w[j], u[i], y[v][i]);
        }
    }
  } else {
    const Row yr(p.y, p.y_bf16, t * p.ld_y, H);
    Raw8 q[V];
#pragma unroll
    for (int v = 0; v < V; ++v) q[v] = yr.load(col[v]);
#pragma unroll
    for (int v = 0; v < V; ++v) yr.values(q[v], y[v]);
  }
  if (p.y_add) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!kAll) aq[v] = y_add.load(col[v]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      y_add.values(aq[v], r[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[v][i] += r[v][i];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!kResid) rq[v] = resid.load(col[v]);
    resid.values(rq[v], r[v]);
  }

  if (p.y) {
    float mul = p.scale;
    if (p.gate && p.gate_col == 0)
      mul *= p.gate_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.gate)[t * p.gate_row])
                         : static_cast<const float*>(p.gate)[t * p.gate_row];
    float inv = 1.0f;
    if (p.post_w) {
      float ss = 0.0f;   // (columns past the row's end hold zeros)
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[v][i], y[v][i], ss);
      inv = rsqrtf(block_sum(ss, part[0], nw) / (float)H + p.eps);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (p.post_w) {
        if (!kAll) oq[v] = post_w.load(col[v]);
        float w[8];
        post_w.values(oq[v], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[v][i] = y[v][i] * inv * (p.w_offset + w[i]);
      }
      if (p.gate && p.gate_col) {
        if (!kAll) gq[v] = gate.load(col[v]);
        float gt[8];
        gate.values(gq[v], gt);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[v][i] *= gt[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) r[v][i] = fmaf(mul, y[v][i], r[v][i]);
      if (col[v] < H) store8(p.resid_out, p.r_bf16, t * p.ld_ro + col[v], r[v]);
    }
  }
  if (p.pre_w) {
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (col[v] < H) {   // (past it: 0 times an infinite scale is NaN)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(r[v][i], r[v][i], ss);
      }
    const float inv = rsqrtf(block_sum(ss, part[1], nw) / (float)H + p.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!kAll) nq[v] = pre_w.load(col[v]);
      float w[8], n[8];
      pre_w.values(nq[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = r[v][i] * inv * (p.w_offset + w[i]);
      if (col[v] < H) store8(p.next, true, t * p.ld_next + col[v], n);
    }
  }
}

template <int V>
hipError_t launch_v(BlockNormArgs a, hipStream_t stream) {
  a.nt = ((a.H / 8 + V - 1) / V + kWave - 1) / kWave * kWave;
  if (a.slot_to_row)
    block_norm_kernel<V, true><<<(unsigned)a.T, a.nt, 0, stream>>>(a);
  else
    block_norm_kernel<V, false><<<(unsigned)a.T, a.nt, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

// Columns a thread holds: 8 while 1024 threads reach over a row (few rows: latency).
hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream) {
  const int per = a.T >= kNormManyRows ? 512 : kNormMaxThreads;   // threads a row at most
  if (a.H <= 8 * (a.T >= kNormManyRows ? 256 : per)) return launch_v<1>(a, stream);
  if (a.H <= 16 * per) return launch_v<2>(a, stream);
  return launch_v<4>(a, stream);
}

}  // namespace nvfp4moe
