// Internal launch interface between the C ABI layer (api.hip) and the kernel files.
// Every launcher only enqueues work on `stream` and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nvfp4moe {

// ---- quantize.hip
size_t quantize_ws_bytes(int64_t B, int64_t R, int64_t C);
// tiled: write codes and scales in the tiled storage of launch_weights_tile (R % 16 == 0).
hipError_t launch_quantize(const void* x, bool x_bf16, int64_t B, int64_t R, int64_t C,
                           const float* g_in, const float* amax_in, bool tiled, uint8_t* packed,
                           uint8_t* scales, float* g_out, void* ws, hipStream_t stream);
size_t fp8_roundtrip_ws_bytes(int64_t n);
hipError_t launch_fp8_roundtrip(const void* x, int64_t n, void* out, void* ws, hipStream_t stream);

// ---- route.hip
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
// Workspace of launch_route_permute: the per-chunk expert counts of the two-launch permutation.
size_t route_permute_ws_bytes(int T, int E, int k);
// The token rows of a W4A16 dispatch: x [T, H] bf16 (after the FP8 E4M3 round trip when fp8)
// prepared for the GEMM into a16 [T, H128] f16 + rexp [T]; rows_ws: dispatch_rows_ws_bytes of
// scratch for the separate round trip (fp8 only).
struct ActPrep {
  const uint16_t* x;
  int H;
  int fp8;
  _Float16* a16;
  int* rexp;
  void* rows_ws;
};
size_t dispatch_rows_ws_bytes(int T, int H, bool fp8);
// Routing and permutation; with prep (nullable) also the token rows' preparation.
hipError_t launch_route_permute(const float* logits, int T, int E, int k, int* topk_ids,
                                float* topk_w, int* expert_offsets, int* sorted_slot,
                                int* slot_to_row, int* active_experts, int* n_active,
                                void* ws, size_t ws_bytes, hipStream_t stream, const ActPrep* prep = nullptr);

// ---- act_prep.hip
// The m-tile list of the large-M path, built by one extra workgroup of the activation prep
// launch (no launch of its own): for the active experts in list order, their m-tiles of bm
// rows; sched_e[i] = expert, sched_r[i] = first row within the expert, sched_n[0] = count (at
// most max_tiles, the length of sched_e and sched_r). max_tiles = 0: no list.
struct MtileSched {
  const int* offsets;
  const int* active;
  const int* n_active;
  int E, bm, max_tiles;
  int* sched_e;
  int* sched_r;
  int* sched_n;
};
// The m-tile list in a launch of its own.
hipError_t launch_mtile_schedule(const MtileSched& sched, hipStream_t stream);
// bf16 rows -> f16 rows scaled by 2^-p (max |x| in [2^14, 2^15)) + p
hipError_t launch_act_prep(const uint16_t* a, int64_t rows, int K, _Float16* a16, int* rexp,
                           const MtileSched& sched, hipStream_t stream);
// NVFP4 rows (codes + E4M3 scales) -> the same f16 layout, decoded exactly (E2M1 * E4M3, the
// global scale stays in the GEMM epilogue); rexp = 0.
hipError_t launch_act_prep_fp4(const uint8_t* packed, const uint8_t* scales, int64_t rows, int K,
                               _Float16* a16, int* rexp, const MtileSched& sched, hipStream_t stream);

// ---- grouped GEMM kernels
struct GemmArgs {
  int w4a4;                        // 0: W4A16 (a16 + rexp), 1: W4A4 (a_packed + a_scales + a_g)
  int a4_staged;                   // W4A4 on the large-M path: 1 = the GEMM decodes the NVFP4 rows
                                   // itself, 0 = it reads their f16 copy (a16) from the activation prep
  const _Float16* a16;             // [a_rows, K] f16, row r scaled by 2^-rexp[r]
  const int* rexp;                 // [a_rows]
  const uint8_t* a_packed;         // [a_rows, K/2]
  const uint8_t* a_scales;         // [a_rows, K/16]
  const float* a_g;                // [1]
  const int* gather_index;         // [rows] or null
  int gather_div;
  const uint8_t* w_packed;         // tiled codes, tiled_codes_bytes(Nw, K) per expert
  const uint8_t* w_scales;         // tiled scales, tiled_scales_bytes(Nw, K) per expert
  const float* w_g;                // [E]
  const int* expert_offsets;       // [E+1]
  const int* active;               // [E]
  const int* n_active;             // [1]
  int E, rows, Nw, K;
  int a_rows;                       // rows of the activation tensor (< 2^31 bytes of it)
  int swiglu;
  void* out;
  int out_bf16;
  float* out_amax;                 // null or [1], zeroed before the GEMM
  const int* sched_e;              // large-M path: m-tile -> expert   (workspace)
  const int* sched_r;              // large-M path: m-tile -> first row (workspace)
  const int* sched_n;              // large-M path: number of m-tiles  (workspace)
  float* partial;                  // large-M split-K: [ksplit, rows, Nw] fp32 partial sums (workspace)
  int ksplit;                      // large-M: K slices (1: no split)
  int unit_alpha;                  // MXFP4: no per-tensor scales (alpha = 1 in the split-K reduce)
  uint8_t* hq_packed;              // MXFP4 SwiGLU: h quantized in the epilogue, [rows, Nw/4] codes
  uint8_t* hq_scales;              //   and [rows, Nw/64] UE8M0 scales (null: out as usual)
  // Fused unpermute + weighted reduce (down GEMM, EPI_NONE, float32 out = Y, no split K):
  const int* comb_slot;            // [rows] sorted_slot: GEMM row -> slot (null: no combine)
  const int* comb_s2r;             // [T * k] slot_to_row
  const float* comb_w;             // [T * k] top-k weights
  int* comb_count;                 // [T * Nw/32] completion counters, zero before the GEMM
  uint16_t* comb_out;              // bf16 [T, Nw]
  int comb_k;
};
// Completion counters of the fused combine: one int per (token, 32 columns), zeroed.
inline size_t comb_count_ints(int T, int Nw) { return (size_t)T * (size_t)(Nw / 32); }
hipError_t launch_zero_i32(int* p, size_t n, hipStream_t stream);
hipError_t launch_gemm_stream(const GemmArgs& a, hipStream_t stream);
// K slices for the small-M path from the sizes alone (1 unless the grid is tiny).
int stream_ksplit(int rows, int E, int Nw, int K);
// Split-K epilogue shared by both GEMM paths: out (and out_amax) from the fixed-order sum of
// the ksplit partial-sum slices in a.partial.
hipError_t launch_splitk_reduce(const GemmArgs& a, hipStream_t stream);
// Tiled weight storage (weights_tile.hip): bytes per [R, C] matrix and the reordering.
size_t tiled_codes_bytes(int64_t R, int64_t C);
size_t tiled_scales_bytes(int64_t R, int64_t C);
hipError_t launch_weights_tile(const uint8_t* packed, const uint8_t* scales, int64_t B, int64_t R, int64_t C,
                               uint8_t* tiled_codes, uint8_t* tiled_scales, hipStream_t stream);
// MXFP4: the same code tiles; UE8M0 scales tiled per (16-row block, 16-chunk window).
size_t mx_tiled_scales_bytes(int64_t R, int64_t C);
hipError_t launch_mx_weights_tile(const uint8_t* packed, const uint8_t* scales, int64_t B, int64_t R, int64_t C,
                                  uint8_t* tiled_codes, uint8_t* tiled_scales, hipStream_t stream);
// MXFP8 (quantize.hip, weights_tile.hip): n elements (n % 32 == 0) -> E4M3 codes [n] + UE8M0
// scales [n/32]; code tiles of 2 KB per (16-row block, chunk), the mx scale tiles.
hipError_t launch_mx8_quantize(const void* x, bool x_bf16, int64_t n, uint8_t* codes, uint8_t* scales,
                               hipStream_t stream);
size_t mx8_tiled_codes_bytes(int64_t R, int64_t C);
hipError_t launch_mx8_weights_tile(const uint8_t* codes, const uint8_t* scales, int64_t B, int64_t R, int64_t C,
                                   uint8_t* tiled_codes, uint8_t* tiled_scales, hipStream_t stream);
// MXFP4 quantizer (quantize.hip): n elements (n % 32 == 0) -> packed [n/2] + UE8M0 scales [n/32].
hipError_t launch_mx_quantize(const void* x, bool x_bf16, int64_t n, uint8_t* packed, uint8_t* scales,
                              hipStream_t stream);
// large-M path: rows per m-tile, the Nw it supports, and the launcher (max_mtiles is the host
// bound ceil(rows / rows_per_mtile) + min(E, rows) on the schedule length).
int large_rows_per_mtile();
bool large_supports(int Nw);
hipError_t launch_gemm_large(const GemmArgs& a, int max_mtiles, hipStream_t stream);
// K slices for the large-M path from the sizes alone (1 when the tiles fill the GPU).
int large_ksplit(int rows, int E, int Nw, int K);
// Waves per large-M workgroup (8, or 4 for small grids), from the sizes alone.
int large_waves(int rows, int E, int Nw);
// MXFP4 W4A4 GEMM on the scaled FP4 MFMA (gemm_mx.hip): m-tile rows, supported Nw, launcher
// (a.w_packed / a.w_scales: MX tiles; a.a_packed / a.a_scales: row-major MXFP4; the m-tile
// list in a.sched_*).
int mx_rows_per_mtile(int bits);   // MX element bits: 4 (MXFP4) or 8 (MXFP8)
bool mx_supports(int Nw);
hipError_t launch_gemm_mx(const GemmArgs& a, int max_mtiles, int bits, hipStream_t stream);
// K slices of the MXFP4 GEMM from the sizes alone (1 unless the grid is under one workgroup per CU).
int mx_ksplit(int max_mtiles, int Nw, int K);
hipError_t launch_zero_f32(float* p, int n, hipStream_t stream);

// ---- few_rows.hip: up to kFewMaxTokens rows
constexpr int kFewMaxTokens = 16;
constexpr int kFewMaxSlots = kFewMaxTokens * kMaxTopK;
constexpr int kFewMaxHidden = 32768;   // H of the layer: at least one row stays in LDS
// What the layer's first launch leaves for its second: the items (expert << 16 | mask of its
// tokens) with the first of their rows in h, and for every row of h its routing weight (NVFP4:
// times the global scale of the expert's second matrix).
struct FewPlan {
  int n_items;
  uint32_t item[kFewMaxSlots];
  uint16_t row0[kFewMaxSlots];
  float weight[kFewMaxSlots];
  int arrived[kFewMaxHidden / 32];   // parts of each tile that are there
};
struct FewArgs {
  const uint16_t* x;      // bf16 [T, K], rows ldx elements apart (matvec, the layer's first launch)
  int64_t ldx;
  int T, K;               // K: columns of the matrices (H, or F in the layer's second launch)
  const uint8_t* codes;   // tiled matrices [Nw, K], one per expert
  const uint8_t* scales;
  const float* g;         // their global scales (NVFP4)
  int Nw;
  int ks_log, item_tok;   // set by the launcher
  uint32_t ppr_inv;
  const void* add;        // matvec: float32 or bf16 [T, n], rows ld_add apart, or null
  int add_bf16;
  int grid;               // workgroups, set by the launcher (the launch's own count lies apart from the arguments)
  int64_t ld_add;
  void* out;              // matvec and the layer's second launch: float32 or bf16
  int out_bf16;
  uint32_t grid_inv;      // set by the launcher: inverse() of grid,
  int64_t ld_out;
  const float* logits;    // layer: [T, E]
  int E, k;
  const float* g_down;    // layer, NVFP4: global scales of the second matrices
  int fp8;                // layer, NVFP4: the rows first take the FP8 E4M3 round trip
  uint32_t tpi_inv;       //   of an item's tiles (first launch), and
  FewPlan* plan;          // layer workspace
  void* h;                // [T * k, F] f16 (NVFP4) or [T * k, 2, F] bf16 (MXFP4: values, and the rest)
  int down_tiles;         // tiles of the second launch
  uint32_t nch_inv;       //   of the chunks of a row (second launch)
  float* part;            // [down_tiles, most_parts, 32 T] sums of a tile that workgroups share
  int most_parts;
  int8_t* hexp;           // NVFP4: [T * k, 8 ceil(F / 128)] exponents of h's blocks of 16 columns
};
hipError_t launch_few_matvec(FewArgs a, bool mx, bool swiglu, hipStream_t stream);
// The layer's second launch: 16-column blocks of a tile, workgroups, and the most that share a tile.
int few_down_blocks(int T, int k, int Nw, int K);
int few_down_workgroups(int T, int k, int Nw, int K);
int few_down_parts(int T, int k, int Nw, int K);
hipError_t launch_few_layer(FewArgs up, FewArgs down, bool mx, hipStream_t stream);

// ---- block_norm.hip
constexpr int kNormMaxH = 32768;
struct BlockNormArgs {
  const void* resid;          // [T, H], rows ld_r apart
  int r_bf16;                 // type of resid and resid_out
  int64_t ld_r;
  const void* y;              // [T, H] or [T * k, H] (slot_to_row), rows ld_y apart, or null
  int y_bf16;
  int64_t ld_y;
  const void* y_add;          // [T, H] added to y, rows ld_ya apart, or null
  int ya_bf16;
  int64_t ld_ya;
  const int* slot_to_row;     // [T * k] or null
  const float* topk_w;        // [T, k]
  int k;
  const void* post_w;         // [H] or null
  const void* pre_w;          // [H] or null
  int w_bf16;
  float w_offset, eps, scale;
  const void* gate;           // element (t, h) at t * gate_row + h * gate_col (0 or 1), or null
  int gate_bf16;
  int64_t gate_row;
  int gate_col;
  int T, H;
  int nt;                     // threads of a workgroup, set by the launcher
  void* resid_out;            // rows ld_ro apart
  int64_t ld_ro;
  void* next;                 // bf16, rows ld_next apart
  int64_t ld_next;
};
hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream);

// ---- reduce.hip
hipError_t launch_unpermute_reduce(const void* y, bool y_bf16, const int* slot_to_row,
                                   const float* topk_w, int T, int k, int H, uint16_t* out,
                                   hipStream_t stream);

// ---- rope_append.hip: rotary positions, and the paged cache's append
// The turn of part of a head: pair i of dims [start, start + rot) by position * freqs[i] radians.
struct RopeTurn {
  const double* freqs;   // [rot / 2], or null: nothing is turned
  int rot, start;
  int interleaved;       // pairs (2i, 2i + 1), else (i, i + rot / 2)
  float magnitude;       // factor of the turned dims
  float sign;            // 1, or -1 for the transposed rotation
};
// Rows of a tensor [T, H, D] whose heads are contiguous: element distances of rows and heads.
struct HeadRows {
  const void* p;
  int64_t row, head;
};
struct RopeArgs {
  HeadRows x, out;
  int bf16;                // type of both (else float32)
  int T, H, D;
  const void* positions;   // [T] int32 or int64
  int pos64;
  RopeTurn turn;
  int copy;                // dims that are not turned are copied (out is not x)
};
hipError_t launch_rope(const RopeArgs& a, hipStream_t stream);

// A batch of sequences whose keys and values lie in pages of `page` tokens.
struct CacheBatchArgs {
  const int* page_table;   // [B, cols], rows ld_table apart: page of a sequence's tokens [c * page, ...)
  int64_t ld_table;
  int cols;
  const int* lengths;      // [B] tokens of each sequence, its new ones among them
  const int* starts;       // [B + 1] row of each sequence's first new token
  int B, T;                // sequences; rows of the tensors of new tokens
  int pages, page, page_log;
};
struct KvAppendArgs {
  HeadRows q, q_out, k, v;   // bf16; q.p null: no queries
  int Hq, Hkv, D;
  CacheBatchArgs batch;
  const void* positions;     // [T] int32 or int64, or null: the tokens' places in their sequences
  int pos64;
  RopeTurn turn;
  void* k_cache;             // [pages, Hkv, page, D]
  void* v_cache;             // [pages, Hkv, D, page]
  int fp8;                   // caches in E4M3, else bf16
  const float* k_scale;      // [Hkv] or null (FP8)
  const float* v_scale;
  int copy;                  // as in RopeArgs, for q
};
hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream);

// ---- kv_attention.hip, kv_attention_few.hip: attention of new tokens over the paged cache
constexpr int kCacheMaxD = 256;
struct KvAttnArgs {
  const uint16_t* q;         // bf16 [T, Hq, D]
  int64_t q_row, q_head;
  uint16_t* out;             // bf16 [T, Hq, D]
  int64_t o_row, o_head;
  int Hq, Hkv, D, G;         // G = Hq / Hkv
  CacheBatchArgs batch;
  const void* k_cache;
  const void* v_cache;
  int fp8;
  const float* k_scale;
  const float* v_scale;
  float scale;               // of the scores
  int window;                // keys that a token sees, itself among them; 0: all
  void* ws;
};
size_t kv_attention_ws_bytes(int T, int B, int Hq, int Hkv, int D);
hipError_t launch_kv_attention(const KvAttnArgs& a, hipStream_t stream);
// its form for tiles of 16 rows (kv_attention_few.hip), and whether the sizes ask for it
bool kv_attention_few_fits(int T, int B, int G);
size_t kv_attention_few_ws_bytes(int Hkv, int D);
hipError_t launch_kv_attention_few(const KvAttnArgs& a, hipStream_t stream);

}  // namespace nvfp4moe
