// Internal declarations shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {

constexpr int kChunk = 64;    // tokens per scan chunk
constexpr int kMaxHead = 128; // largest d_k / d_v

// Parameters of one replay (or chunk-operator) launch on the fp32 CUDA-core path.
struct SimtParams {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  const int32_t* cu;  // nullptr: one sequence of total_tokens
  const float* S0;
  void* O;
  float* S_out;   // value rows: [n_seqs][h_v][d_v][d_k]
  float* T_out;   // chunk-operator mode: [n_seqs][h_v][d_k][d_k]
  int n_seqs, total_tokens, h_k, h_v, d_k, d_v;
  int augmented;  // 1: state carries d_k extra transition rows (chunk operator)
  int l2norm;
  int write_O;
  int scalar_decay;  // 1: scalar per-token transition (no rank-1 projection term)
  float scale;
  int* status;    // sticky device status word
  unsigned char* rec;  // optional per-(chunk, v-head) records of the chunk-shared quantities (scratch)
};

// fp32 record of the chunk-shared quantities of one (chunk, v-head), written by the fp32 path's
// prep kernel: M = (I + A)^{-1} [64][64] (row t, column s), P [64][64] (only when outputs are
// wanted), then per token t: gamma_t, exp(G_last - G_t), beta_t, rk_t (key norm factor), rq_t
// (query norm factor times scale).  Offsets in floats.
constexpr int REC_M = 0, REC_P = 4096, REC_GAM = 8192, REC_WEND = 8256, REC_BETA = 8320, REC_RK = 8384,
              REC_RQ = 8448, REC_FLOATS = 8512;

cudaError_t launch_replay_simt(const SimtParams& p, int bf16, cudaStream_t stream);
// Scratch bytes of the two-kernel CUDA-core path (chunk-parallel prep, then the row-slice scan).
size_t simt_records_bytes(int n_seqs, int total_tokens, int h_v);
// The same computation as launch_replay_simt, with the chunk-shared work (norms, gates, Gram,
// (I + A)^{-1}) done once per (chunk, v-head) by a prep kernel into `workspace` first.
cudaError_t launch_replay_simt_two_pass(SimtParams p, int bf16, void* workspace, size_t bytes, cudaStream_t stream);

// Tensor-core path (bf16 inputs, d_k = d_v = 128, total_tokens > 0): a chunk-parallel
// prep kernel writes per-(chunk, v-head) records into `workspace`, then the scan
// kernel walks each tail.  workspace_bytes must be >= replay_tc_workspace_bytes().
bool replay_tc_supported(const SimtParams& p);
size_t replay_tc_workspace_bytes(int n_seqs, int total_tokens, int h_v);
cudaError_t launch_replay_tc(const SimtParams& p, void* workspace, size_t workspace_bytes, cudaStream_t stream);
int replay_tc_rows(int n_seqs, int h_v);

constexpr int kMaxCompose = 256;  // largest K of one gdn_compose call

// Passed by value: the K device pointers travel in the kernel parameters.
struct ComposeParams {
  const float* T[kMaxCompose];
  const float* Slocal[kMaxCompose];
  const float* S_in;
  float* S_out;
  int* status;  // sticky device status word (bounded waits that give up report GDN_ERR_TIMEOUT)
  unsigned long long wait_ns;  // limit of each bounded wait (0: give up unless already complete)
  int K, h, d_k, d_v;
};

cudaError_t launch_compose_simt(const ComposeParams& p, cudaStream_t stream);
// Tensor-core composition (split tf32, fp32 accuracy) for d_k = d_v = 128 and K >= 1.
bool compose_tc_supported(const ComposeParams& p);
cudaError_t launch_compose_tc(const ComposeParams& p, cudaStream_t stream);

// The driver's tensor-map encoder (null if unavailable).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
// Tensor map of a 2D bf16 view [rows][cols] (cols contiguous) with boxes of 64 columns x
// box_rows rows, 128-byte swizzle (the tile layout the tensor-core operands use); false if the
// driver's encoder is unavailable or rejects the view.
bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows);
// The same for a 2D fp32 view: boxes of 32 columns (128 bytes) x box_rows rows.
bool make_map_f32(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows);

// Operator-form state-only scan (bf16 inputs, d_k = d_v = 128, 32-row slices) over the records
// of the tensor-core prep kernel written with the Z factor (see state_tc.cu).
struct StateParams {
  const int32_t* cu;
  const int32_t* order;  // tails longest first, or null
  const float* S0;
  const unsigned char* rec;
  float* S_out;
  int* status;
  int n_seqs, total_tokens, h_k, h_v;
};
cudaError_t launch_state_tc(const CUtensorMap& mk, const CUtensorMap& mv, const StateParams& sp, bool overlap_prep,
                            cudaStream_t stream);

// Tensor-core state-only scan of the fp32 path (d_k = d_v = 128, fp32 or bf16 inputs, no
// outputs), over the records already written into p.rec: the state (augmented or not) in
// 128-row slices, at fp32 accuracy.
bool chunkop_tc_supported(const SimtParams& p, int bf16);
cudaError_t launch_chunkop_tc(const SimtParams& p, int bf16, cudaStream_t stream);

// Linear attention with a decay for each head over packed prompts (gdn_linear_attn).
struct LinearParams {
  const void* q;
  const void* k;
  const void* v;
  const float* log_decay;  // [h_v]
  const int32_t* cu;
  const float* S0;  // or null
  void* O;
  float* S_out;
  int* status;
  int n_seqs, total_tokens, h_k, h_v, d_k, d_v;
  int write_O;
  float scale;
};
// Scratch that a call needs on the current device (may be 0), and the call.
cudaError_t linear_workspace_bytes(const LinearParams& p, int bf16, size_t* bytes);
cudaError_t launch_linear(const LinearParams& p, int bf16, void* workspace, cudaStream_t stream);

// S <- lambda^n S + D of a carried state, lambda = exp(g).  A factor near 1 stored in fp32 is off by
// up to 2^-25, always the same way, and a long prompt multiplies by it hundreds of times; the step
// S + (lambda^n - 1) S is off by 2^-24 |lambda^n - 1| instead, plus the sum's own unbiased rounding.
// Below 1/2 the factor itself is exact enough (and S + (f - 1) S would cancel).
struct DecayStep {
  float f, f1;
  bool near1;
  __device__ __forceinline__ float operator()(float s, float d) const {
    return near1 ? fmaf(s, f1, s + d) : fmaf(s, f, d);
  }
};
__device__ __forceinline__ DecayStep decay_step(float g, int n) {
  DecayStep r;
  r.f = expf((float)n * g);
  r.f1 = expm1f((float)n * g);
  r.near1 = r.f1 >= -0.5f;
  return r;
}

// Recurrent form on a pool of states (gdn_decode).
enum : int { kDelta = 0, kScalarDecay = 1, kHeadDecay = 2 };
struct DecodeParams {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;      // null for kHeadDecay
  const int32_t* slots;   // or null: request i on slot i
  const int32_t* counts;  // or null: the whole window
  float* S;               // [n_slots][h_v][d_v][d_k]
  void* O;
  int* status;
  int n, window, n_slots, h_k, h_v, d_k, d_v;
  int v_per_k;  // h_v / h_k
  int family, l2norm, state_only, keep;
  float scale;
};
cudaError_t launch_decode(const DecodeParams& p, int bf16, cudaStream_t stream);

// Verification of drafted tokens (gdn_verify_draft).
struct VerifyParams {
  const void* target;
  const void* draft;          // or null
  const int32_t* drafted;     // [n][n_draft]
  const int32_t* draft_lens;  // or null
  const float* uniforms;      // [n][n_draft + 1]
  int32_t* counts;            // [n]
  int32_t* tokens;            // [n][n_draft + 1]
  int* status;
  int64_t target_stride, draft_stride;  // elements between consecutive rows
  int n, n_draft, vocab;
};
cudaError_t launch_verify(const VerifyParams& p, int bf16, cudaStream_t stream);

// Paged key-value cache (gdn_kv_append, gdn_paged_attn).
struct PagedParams {
  const void* q;
  const void* k;  // gdn_kv_append: the new keys and values; gdn_paged_attn: the pages
  const void* v;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* cu;  // or null: total / n tokens each
  void* O;            // gdn_kv_append: the rotated queries
  float* lse;         // or null
  void* k_pages;      // gdn_kv_append
  void* v_pages;
  const float* inv_freq;
  const int32_t* positions;  // or null
  int* status;
  int64_t table_stride, q_stride, k_stride, v_stride, k_page, k_token, k_head, v_page, v_token, v_head;
  int n, total, max_q, h_q, h_kv, group, d, page_shift, n_pages, width, window;
  float scale;
  int rotary, neighbours, n_axes, sections[GDN_MAX_AXES];
};
cudaError_t launch_kv_append(const PagedParams& p, int bf16, cudaStream_t stream);
// Scratch that a call needs on the current device, and the call.
cudaError_t paged_workspace_bytes(const PagedParams& p, int bf16, size_t* bytes);
cudaError_t launch_paged_attn(const PagedParams& p, int bf16, void* workspace, cudaStream_t stream);

// Beams (gdn_beam_select, gdn_beam_reorder).
constexpr int kMaxBeams = 64;  // beams of a request, and continuations that are selected
struct BeamParams {
  const void* logits;
  const float* scores;  // [n][beams]
  float* scores_out;    // [n][best]
  int32_t* parents;
  int32_t* tokens;
  int64_t stride;       // elements between consecutive rows of logits
  int n, beams, best, vocab;
};
cudaError_t beam_workspace_bytes(const BeamParams& p, size_t* bytes);
cudaError_t launch_beam_select(const BeamParams& p, int bf16, void* workspace, cudaStream_t stream);
struct ReorderParams {
  unsigned char* pool;
  const int32_t* slots;    // [n][beams]
  const int32_t* parents;  // [n][beams]
  int32_t* slots_out;      // [n][beams]
  int* status;
  int64_t row_bytes, slot_stride, layer_stride;  // bytes
  int n, beams, n_slots, layers;
};
cudaError_t launch_beam_reorder(const ReorderParams& p, cudaStream_t stream);

// Sticky status word of the current device (device pointer).
int* device_status_word();

// Helpers of the allocation-free replay entry point (defined in gdn_api.cu).
int check_replay_args(const gdn_dims* dims, const void* q, const void* k, const void* v, const float* g,
                      const float* beta, const int32_t* cu_seqlens, const float* S0, void* O_out, float* S_out,
                      SimtParams* p, bool* nothing_to_do);
int report_error(int code, const char* message);
// The event set by gdn_set_stage_event on this thread (nullptr if none); clears it.
void* take_stage_event();
// The wait limit set by gdn_set_wait_limit_ns on this thread (else the 2 s default); clears it.
unsigned long long take_wait_limit_ns();

}  // namespace gdn
