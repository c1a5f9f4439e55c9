// The norms around a block with its gate and residual scale (gfx950), in one pass over the rows:
//   u    = y                                      y / sqrt(mean(y^2) + eps) * (o + post_w)  with post_w
//   r'   = r + scale * gate * u
//   next = bf16( r' / sqrt(mean(r'^2) + eps) * (o + pre_w) )                               with pre_w
// y is the block's output, or the experts' rows with their weights: y_t = sum_j w[t, j] Y[row of
// slot (t, j)] in ascending j (the unpermute-reduce, whose bf16 output then never exists); y_add
// (a shared expert's output) is added to either. Without
// y only next is written (the norm before the first block).
//
// Memory-bound: y (k rows of it for the experts' form), r and a full gate are read once, r' and
// next written once; everything between stays in registers. One workgroup a row: a thread holds
// V groups of 8 consecutive columns (16- and 32-byte accesses), the two sums of squares meet in
// LDS (float32: at most 32 squares a thread, then a tree over lanes and waves). Next is computed from r' in
// float32, before r' is rounded to its stored type.
#include "common.h"
#include "kernels.h"

namespace nvfp4moe {

namespace {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormBatch = 4;      // experts' rows requested together
constexpr int kNormManyRows = 256; // rows from which a thread holds more columns

// Eight consecutive values as float32 (o: element offset).
__device__ __forceinline__ void load8(const void* p, bool bf16, int64_t o, float (&v)[8]) {
  if (bf16) {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + o);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + o);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + o + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
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

// Sum over the workgroup, in every thread; part: kNormMaxThreads / 64 floats of LDS of its own.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  const int nw = blockDim.x / kWave;
  if (nw == 1) return v;
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < nw; ++w) s += part[w];
  return s;
}

template <int V, bool ROWS>
__global__ __launch_bounds__(kNormMaxThreads) void block_norm_kernel(const BlockNormArgs p) {
  __shared__ float part[2][kNormMaxThreads / kWave];
  const int64_t t = blockIdx.x;
  const int H = p.H;
  int col[V];
#pragma unroll
  for (int v = 0; v < V; ++v) col[v] = ((int)threadIdx.x + v * (int)blockDim.x) * 8;

  float r[V][8], y[V][8];
  if (ROWS) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[v][i] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += kNormBatch) {
      int64_t row[kNormBatch];
      float w[kNormBatch];
#pragma unroll
      for (int j = 0; j < kNormBatch; ++j) {   // (the row is the workgroup's: scalar loads)
        const bool in = j0 + j < p.k;
        row[j] = in ? (int64_t)ld_const(p.slot_to_row, t * p.k + j0 + j) : 0;
        w[j] = in ? ld_const(p.topk_w, t * p.k + j0 + j) : 0.0f;
      }
      float q[kNormBatch][V][8];
#pragma unroll
      for (int j = 0; j < kNormBatch; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (j0 + j < p.k && col[v] < H) load8(p.y, p.y_bf16, row[j] * p.ld_y + col[v], q[j][v]);
#pragma unroll
      for (int j = 0; j < kNormBatch; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (j0 + j < p.k && col[v] < H) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[v][i] = fmaf(w[j], q[j][v][i], y[v][i]);
          }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (p.y && col[v] < H) load8(p.y, p.y_bf16, t * p.ld_y + col[v], y[v]);
  }
  if (p.y_add) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (col[v] < H) {
        load8(p.y_add, p.ya_bf16, t * p.ld_ya + col[v], r[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[v][i] += r[v][i];
      }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (col[v] < H) load8(p.resid, p.r_bf16, t * p.ld_r + col[v], r[v]);

  if (p.y) {
    float mul = p.scale;
    if (p.gate && p.gate_col == 0)
      mul *= p.gate_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.gate)[t * p.gate_row])
                         : static_cast<const float*>(p.gate)[t * p.gate_row];
    float inv = 1.0f;
    if (p.post_w) {
      float ss = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (col[v] < H) {
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(y[v][i], y[v][i], ss);
        }
      inv = rsqrtf(block_sum(ss, part[0]) / (float)H + p.eps);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (col[v] < H) {
        if (p.post_w) {
          float w[8];
          load8(p.post_w, p.w_bf16, col[v], w);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[v][i] = y[v][i] * inv * (p.w_offset + w[i]);
        }
        if (p.gate && p.gate_col) {
          float gt[8];
          load8(p.gate, p.gate_bf16, t * p.gate_row + col[v], gt);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[v][i] *= gt[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) r[v][i] = fmaf(mul, y[v][i], r[v][i]);
        store8(p.resid_out, p.r_bf16, t * p.ld_ro + col[v], r[v]);
      }
  }
  if (p.pre_w) {
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (col[v] < H) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(r[v][i], r[v][i], ss);
      }
    const float inv = rsqrtf(block_sum(ss, part[1]) / (float)H + p.eps);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (col[v] < H) {
        float w[8], n[8];
        load8(p.pre_w, p.w_bf16, col[v], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = r[v][i] * inv * (p.w_offset + w[i]);
        store8(p.next, true, t * p.ld_next + col[v], n);
      }
  }
}

template <int V>
hipError_t launch_v(const BlockNormArgs& a, hipStream_t stream) {
  const int nt = ((a.H / 8 + V - 1) / V + kWave - 1) / kWave * kWave;
  if (a.slot_to_row)
    block_norm_kernel<V, true><<<(unsigned)a.T, nt, 0, stream>>>(a);
  else
    block_norm_kernel<V, false><<<(unsigned)a.T, nt, 0, stream>>>(a);
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
