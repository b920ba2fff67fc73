// Host-side launchers shared between the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// Device error word (first error wins); lives at offset 0 of the workspace.
enum DevErr : int { kDevOk = 0, kDevTimeout = 1, kDevBadIndex = 2 };

struct Shape {
  int64_t T;
  int H, E, K, F, C;   // C <= 0: no capacity limit
  int dtype;           // MOE_F32 | MOE_BF16
  uint32_t flags;
  float inv_tau;       // 1 / router softmax temperature
  int64_t S() const { return T * (int64_t)K; }
  size_t esize() const { return dtype == MOE_BF16 ? 2 : 4; }
};

// The kernels' view of a validated layer description (temperature -> 1/tau).
Shape shape_of(const moe_desc& d);

// Number of SMs of the current device (cached per device).
int sm_count();

// Launch with programmatic dependent launch allowed (the kernel waits for its
// predecessor itself, see pdl_enter) and an optional cluster size.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_kernel(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                 unsigned cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Stage-boundary events of moe_layer_forward (set by moe_profile_events; no-op
// when unset).  Marks: 0 start, 1 router, 2 dispatch, 3 first product,
// 4 second product, 5 combine.
enum ProfMark { kMarkStart = 0, kMarkRouter, kMarkDispatch, kMarkFirst, kMarkSecond, kMarkCombine, kMarks };
void prof_mark(int mark, cudaStream_t st);

// Row-major bf16 matrix [rows, cols] as a 2D TMA tensor map with a box of
// 64 columns (128 bytes, 128-byte swizzle) x box_rows rows; false on failure.
bool tma_map_bf16(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint32_t box_rows);

// Row-major bf16 [d2, rows, cols] as a 3D tensor map with a box of 1 x box_rows
// x 64 columns (128-byte swizzle): what lies outside a [rows, cols] matrix
// reads as zero and is not written.
bool tma_map_bf16_3d(CUtensorMap* m, const void* ptr, uint64_t d2, uint64_t rows, uint64_t cols, uint32_t box_rows);

// The same for 16-bit elements whose rows are `pitch` and matrices `plane`
// elements apart (multiples of 8); boxes of other than 64 columns are not
// swizzled.
bool tma_map_16bit_3d(CUtensorMap* m, const void* ptr, uint64_t d2, uint64_t rows, uint64_t cols, uint64_t pitch,
                      uint64_t plane, uint32_t box_rows, uint32_t box_cols = 64);

// ---------------------------------------------------------------- router
// Upper bound of the rows of per-block probability partial sums the router
// writes (workspace sizing), and the rows the chosen router writes.
int64_t router_partials(const Shape& s);
bool router_small(const Shape& s);   // one-cluster router for decode-sized bf16 batches
int64_t router_partial_rows(const Shape& s);
bool router_on_tensor_cores(const Shape& s);
int router_tc_split(const Shape& s);   // CTAs the tensor-core router splits the hidden dimension over (1 or 2)
// tile_hist (nullable): [ceil(T/128), E] count of each 128-token tile's
// chosen experts, in slot order blocks of 128*K slots.
cudaError_t launch_router_tc(const Shape& s, const void* x, const void* Wg, const float* gate_bias,
                             float* logits, int32_t* ids, float* w, float* psum_part,
                             int32_t* tile_hist, int* err, cudaStream_t st);
constexpr int kRouterTileTokens = 128;
cudaError_t launch_router(const Shape& s, const void* x, const void* Wg, const float* gate_bias,
                          float* logits, int32_t* ids, float* w, float* psum_part, int* err,
                          cudaStream_t st, int32_t* tile_hist = nullptr);
// psum[e] = sum over partial rows in order.
cudaError_t launch_psum_reduce(const Shape& s, const float* psum_part, float* psum, cudaStream_t st);

// ---------------------------------------------------------------- dispatch
int64_t dispatch_blocks(const Shape& s);
int dispatch_block_slots(const Shape& s);
bool dispatch_small(const Shape& s);
int dispatch_launches(const Shape& s, bool hist_ready);   // kernels launch_dispatch issues (S > 0)   // one-block dispatch (launch_dispatch picks it itself)
struct DispatchOut {
  int32_t* count;      // [E]
  int32_t* offs;       // [E+1]
  int32_t* src;        // [rows]
  int32_t* pos;        // [S]
  int32_t* dropped;    // [1] or null
  int32_t* blk_hist;   // [nblk * E] scratch
  int32_t* blk_base;   // [nblk * E] scratch
  // optional extras folded into the scan kernel
  const float* psum_part;  // partial rows or null
  bool hist_ready;         // blk_hist already holds the router's per-tile counts
  float* psum;             // [E] or null
  float* aux;              // [1] or null (needs psum_part)
  int32_t* count_copy;     // [E] or null
  int32_t* dropped_copy;   // [1] or null
  int32_t* sched;          // [sched_words] the expert GEMMs' counters, zeroed here, or null
};
cudaError_t launch_dispatch(const Shape& s, const int32_t* ids, const void* x, void* x_perm,
                            const DispatchOut& o, int* err, cudaStream_t st);

// drop_tokens=False: fin [S] = each slot's expert after the over-capacity
// slots (pos < 0 in the capacity-limited dispatch with row offsets offs) have
// moved to their token's next-best expert with room, or -1; scores [T, E] are
// the router's; pend, choice: [S] and alts: [T, E] scratch.  dropped
// (nullable): slots left without an expert.  Two launches.
cudaError_t launch_reroute(const Shape& s, const float* scores, const int32_t* ids, const int32_t* pos,
                           const int32_t* offs, int32_t* fin, int32_t* pend, int32_t* choice, uint8_t* alts,
                           int32_t* dropped, int32_t* dropped_copy, cudaStream_t st);

// ---------------------------------------------------------------- expert FFN
// The SM-pair expert GEMMs' counters: two tile counters, then one ready
// counter per 256-row block of the kept rows (at most rows / 256 + E + 1).
inline int64_t sched_words(int64_t rows, int E) { return 2 + rows / 256 + E + 1; }
// Decode-sized batches that run the weight-streaming kernels, and those of
// them that run both products in one launch (its per-expert counters are
// sched[2 .. 2 + E)).
bool stream_ffn_eligible(const Shape& s);
bool stream_fused(const Shape& s);
// The weighted combine folded into the second product's epilogue (K <= 2,
// SM-pair kernels): row r adds w[src[r]] * y to acc[src[r] / K] (fp32,
// zeroed beforehand) instead of storing y.
struct CombineInto {
  const int32_t* src;
  const float* w;
  float* acc;
};
bool combine_fusable(const Shape& s, int64_t max_rows);
// The first product's token rows read from x by the slot list (kept row r:
// x row src[r] / K) instead of from x_perm (SM-pair kernels only).
struct GatherRows {
  const void* x;
  const int32_t* src;
};
// sched: sched_words(max_rows, E) zeroed ints (the SM-pair kernel's counters)
cudaError_t launch_ffn(const Shape& s, int64_t max_rows, const void* x_perm, const int32_t* offs,
                       const void* W1, const float* b1, const void* W2, const float* b2,
                       void* h_perm, void* y_perm, int* err, int32_t* sched, cudaStream_t st,
                       const CombineInto* comb = nullptr, const GatherRows* gather = nullptr);

// ---------------------------------------------------------------- one-launch decode layer
// bf16 batches of at most 16 tokens whose rows, score table and weight ring
// fit one CTA's shared memory, unless the flags ask for the separate steps.
bool decode_layer_eligible(const Shape& s);
// workspace: [pieces][T][E] fp32 partial gate scores, and the counters
size_t decode_part_floats(const Shape& s);
int decode_ctr_words(const Shape& s);
struct DecodeIO {
  const void* x;
  const void* Wg;
  const float* gate_bias;
  const void* W1;
  const float* b1;
  const void* W2;
  const float* b2;
  void* out;
  float* part;
  int* ctr;
  void* h;      // [kept rows, F]
  void* y;      // [kept rows, H]
  int32_t* count;
  int32_t* count_copy;
  int32_t* dropped;
  int32_t* dropped_copy;
  float* psum;
  float* aux;
  int* err;
};
// Two launches: the counters zeroed, then the layer.
cudaError_t launch_decode_layer(const Shape& s, const DecodeIO& io, cudaStream_t st);

// ---------------------------------------------------------------- combine / aux
cudaError_t launch_combine(const Shape& s, const void* y_perm, const int32_t* pos, const float* w,
                           void* out, cudaStream_t st);
cudaError_t launch_aux(const Shape& s, const float* psum, const int32_t* count, float* loss,
                       cudaStream_t st);
// acc [T, H] fp32 = 0, and out [T, H] = bf16(acc) (the fused combine's two ends)
cudaError_t launch_zero_acc(const Shape& s, float* acc, cudaStream_t st);
cudaError_t launch_acc_to_out(const Shape& s, const float* acc, void* out, cudaStream_t st);
// ---------------------------------------------------------------- training
cudaError_t launch_combine_backward(const Shape& s, const void* dout, const void* y_perm, const int32_t* pos,
                                    const float* w, void* dy_perm, float* dw, cudaStream_t st);
cudaError_t launch_dispatch_backward(const Shape& s, const void* dx_perm, const int32_t* pos, const void* add,
                                     void* dx, cudaStream_t st);
// The expert FFN's gradient: what moe_expert_ffn_backward is given (the
// results nullable, one by one).
struct FfnBackward {
  const void* x_perm;
  const void* h_perm;
  const void* dy_perm;
  const int32_t* offs;
  const void* W1;
  const float* b1;
  const void* W2;
  void* dx_perm;
  void* dW1;
  float* db1;
  void* dW2;
  float* db2;
};
// da: [max_rows, F or 2F] fp32 scratch
cudaError_t launch_ffn_backward_simt(const Shape& s, int64_t max_rows, const FfnBackward& b, float* da,
                                     cudaStream_t st);
// bf16 on SM pairs.  da: [max_rows, F or 2F] bf16, stash:
// backward_stash_floats, part: [8 * backward_blocks(max_rows, E), F or 2F]
// fp32, tails: backward_tail_bytes (N = F or 2F), 128-byte aligned: scratch.
size_t backward_stash_floats();
int64_t backward_blocks(int64_t rows, int E);
size_t backward_tail_bytes(int E, int H, int N, int F);
cudaError_t launch_ffn_backward_tc(const Shape& s, int64_t max_rows, const FfnBackward& b, void* da, float* stash,
                                   float* part, void* tails, int* err, cudaStream_t st);
cudaError_t launch_adamw(const moe_adamw_tensor* tensors, int count, int grad_dtype, int state_bits,
                         const moe_adamw_params& h, const float* grad_scale, const int32_t* skip, cudaStream_t st);


// The load-balancing loss and the router's gradient.  blocks: partial sums of
// the tokens' kernels; the products' scratch follows from the shape.
int64_t balance_partials(const Shape& s);
int64_t dlogits_partials(const Shape& s);
struct BalanceOut {
  float* psum;
  int32_t* count;
  int32_t* tokens;
  float* loss;
};
// part_p: [balance_partials, E] floats, part_c: [balance_partials, E + 1] ints
cudaError_t launch_balance(const Shape& s, const float* logits, const int32_t* ids, const uint8_t* mask,
                           const BalanceOut& o, float* part_p, int32_t* part_c, int* err, cudaStream_t st);
struct RouterBackward {
  const void* x;
  const void* Wg;
  const float* logits;
  const int32_t* ids;
  const float* dw;
  const float* dloss;
  const int32_t* count;
  const int32_t* tokens;
  const uint8_t* mask;
  float* dlogits;
  float* dWg;
  float* dbias;
  void* dx;
};
// dl: router_scratch_bytes: the scores' gradient, [T, E] fp32, or in bf16
// parts; part_b: [dlogits_partials, E] floats, part_w: router_weight_partials
// floats
bool router_gate_on_tensor_cores(const Shape& s);
size_t router_scratch_bytes(const Shape& s);
int64_t router_weight_partials(const Shape& s);
// The gate's products on the tensor cores, and the sum of part_b's rows_b rows
// into dbias.  panels: [T, gate_panel_cols] bf16 and alive as
// dlogits_kernel writes them.
int gate_panel_cols(int E);
bool gate_skips_tiles(int E);   // whether the products leave out tiles by their flags
int64_t gate_part_floats(const Shape& s);
cudaError_t launch_gate_tc(const Shape& s, const RouterBackward& b, const void* panels, const uint8_t* alive,
                           float* part, const float* part_b, int rows_b, int* err, cudaStream_t st);
cudaError_t launch_router_backward(const Shape& s, const RouterBackward& b, void* dl, float* part_b, float* part_w,
                                   int* err, cudaStream_t st);

// Orthogonalised updates.  With `tensors` of one matrix each way round in
// `raw`: moe_orthogonalize; else a Muon step.  stall: testing, barriers wait for
// an arrival that nobody makes.
struct OrthogonalRaw {
  const void* x;
  int x_dtype;
  void* out;
  int out_dtype;
};
size_t orthogonal_workspace(const moe_muon_tensor* tensors, int count);
cudaError_t launch_orthogonal(const moe_muon_tensor* tensors, int count, int grad_dtype, const moe_muon_params& h,
                              const OrthogonalRaw* raw, const float* grad_scale, const int32_t* skip, bool stall,
                              void* ws, cudaStream_t st);

// The statistics of a layer run in pieces of tokens: count[e] and psum[e]
// summed over the n pieces in order, then the loss of the whole batch (s.T
// tokens); count_copy, aux and dropped (0: no capacity) are nullable.
cudaError_t launch_merge_stats(const Shape& s, const int32_t* count_parts, const float* psum_parts, int n,
                               int32_t* count, float* psum, int32_t* count_copy, float* aux, int32_t* dropped,
                               cudaStream_t st);

}  // namespace moe
