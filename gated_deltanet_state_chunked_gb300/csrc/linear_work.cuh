// Work list of gdn_linear_attn, shared by its tensor-core (bf16) and CUDA-core (fp32) kernels.
//
// An item is one (segment of a sequence, v-head).  A sequence longer than `seg_tokens` is cut into
// segments, so that a few long prompts fill the GPU: the segments' own states first (from zero), then
// their entering states (linear_carry_kernel), then every segment with its outputs.  With several
// sequences linear_plan_kernel lists the segments, longest first, once per call.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_internal.cuh"

namespace gdn {

// One entry of the plan: a segment of a sequence.  seq < 0: none.
struct Segment {
  int seq, seg, n_seg, t_begin, len, local, pad0, pad1;
};
// The entering states of a cut sequence's segments are found sequence by sequence.
struct CutSeq {
  int seq, n_seg, local, last_len;
};

struct LinearWork {
  const void* q;
  const void* k;
  const void* v;
  const float* log_decay;
  const int32_t* cu;
  const float* S0;
  float* local;         // [cut segments][h_v][d_v][d_k]: the segments' own, then entering states
  const Segment* list;  // the launch's segments, or null: one sequence, its segments in order
  const CutSeq* cuts;   // linear_carry_kernel: cut sequences, or null: one sequence
  void* O;
  float* S_out;
  int* status;
  int n_seqs, total_tokens, h_k, h_v, d_k, d_v;
  int seg_tokens;   // INT_MAX: sequences are not cut
  int cut_units;    // segments that `local` has room for
  int local_only;   // the segments' own states for a launch with outputs: the last one is not needed
  int early;        // the launch may start before the kernel ahead of it ends, and waits for it before
                    // it reads the list (where there is one) or a state in `local`
  float scale;
};

__device__ __forceinline__ int segments_of(int len, int seg_tokens) {
  return len <= seg_tokens ? 1 : (len - 1) / seg_tokens + 1;
}
// Segment `u` of a call with one sequence (seq = -1: there is no such segment).
__device__ __forceinline__ Segment only_segment(const LinearWork& p, int u) {
  Segment s = {};
  const int a = p.cu[0], b = p.cu[1];
  s.seq = -1;
  if (a >= 0 && b >= a && b <= p.total_tokens) {
    s.n_seg = segments_of(b - a, p.seg_tokens);
    if (u < s.n_seg) {
      s.seq = 0;
      s.seg = s.local = u;
      s.t_begin = a + u * (s.n_seg > 1 ? p.seg_tokens : 0);
      s.len = min(p.seg_tokens, b - s.t_begin);
    }
  }
  return s;
}
// Where an item's state comes from (null: zero) and goes to: the index of a state in S_out or in
// `local`, -1: nowhere.  out: a launch with outputs.
struct ItemState {
  const float* S_in;
  int dst, to_local;
};
__device__ __forceinline__ ItemState item_state(const LinearWork& p, const Segment& s, int h, bool out) {
  const size_t dd = (size_t)p.d_v * p.d_k, whole = ((size_t)s.seq * p.h_v + h) * dd, part = ((size_t)s.local * p.h_v + h) * dd;
  const bool cut = s.n_seg > 1, final = !cut || (out && s.seg + 1 == s.n_seg);
  ItemState r;
  r.S_in = cut ? (out ? p.local + part : nullptr) : p.S0 ? p.S0 + whole : nullptr;
  r.to_local = !final;
  r.dst = final ? s.seq * p.h_v + h : out ? -1 : s.local * p.h_v + h;
  return r;
}

// The item kernels: every unit of `p` (segments, in the order of the list) times every v-head.
cudaError_t launch_linear_tc_items(const LinearWork& p, bool out, int units, cudaStream_t stream);
cudaError_t launch_linear_simt_items(const LinearWork& p, bool out, int units, cudaStream_t stream);

}  // namespace gdn
