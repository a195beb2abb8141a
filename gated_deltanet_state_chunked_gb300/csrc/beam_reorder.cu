// gdn_beam_reorder: the rows of a pool follow their beams.
#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kReorderNT = 256;
constexpr int64_t kPiece = 64 * 1024;  // bytes of a row that one CTA copies

// Grid: (requests * beams, pieces of a row, layers).  A beam's first child keeps its parent's slot; the k-th of the
// other beams takes the slot of the k-th beam without children and gets a copy of its parent's row.  A row
// that is written had no children, so nothing reads it, and the copies need no order among them.  Every
// CTA finds the plan of its request by itself (two short trips to L2, beside 64 KB to copy).  Bound by HBM: 512 beams of 2 MB,
// 222 of them copied, 121 us (7.7 TB/s of copies; a row that several children copy comes from L2 after the first).
__global__ void __launch_bounds__(kReorderNT) beam_reorder_kernel(ReorderParams p) {
  __shared__ int slot[kMaxBeams], parent[kMaxBeams], keeps[kMaxBeams], childless[kMaxBeams], free_rank[kMaxBeams];
  const int tid = threadIdx.x, req = blockIdx.x / p.beams, beam = blockIdx.x - req * p.beams;
  const int64_t first = (int64_t)req * p.beams;
  if (tid < p.beams) {
    slot[tid] = p.slots[first + tid];
    parent[tid] = p.parents[first + tid];
  }
  __syncthreads();
  const bool reports = blockIdx.y == 0 && blockIdx.z == 0;
  if (slot[0] < 0) {  // padding
    if (reports && tid == 0) p.slots_out[first + beam] = -1;
    return;
  }
  bool bad = false;
  if (tid < p.beams) {
    const int par = parent[tid];
    bad = (unsigned)slot[tid] >= (unsigned)p.n_slots || par >= p.beams;
    bool keep = par >= 0, none = true;
    for (int j = 0; j < p.beams; ++j) {
      keep = keep && !(j < tid && parent[j] == par);
      none = none && parent[j] != tid;
      bad = bad || (j < tid && slot[j] == slot[tid]);
    }
    keeps[tid] = keep;
    childless[tid] = none;
  }
  __syncthreads();
  const bool copies = !keeps[beam] && parent[beam] >= 0;
  if (!copies && !reports) return;
  // a slot that an earlier request names too
  for (int64_t i = tid; i < first; i += kReorderNT) {
    const int s = p.slots[i];
    if (s >= 0 && p.slots[i - i % p.beams] >= 0)  // (not those of padding)
      for (int j = 0; j < p.beams; ++j) bad = bad || slot[j] == s;
  }
  if (__syncthreads_or(bad)) {
    if (reports && tid == 0) {
      p.slots_out[first + beam] = -1;
      atomicExch(p.status, GDN_ERR_SHAPE);
    }
    return;
  }
  if (tid < p.beams && childless[tid]) {
    int rank = 0;
    for (int j = 0; j < tid; ++j) rank += childless[j];
    free_rank[rank] = tid;
  }
  __syncthreads();
  int target;
  if (keeps[beam]) {
    target = slot[parent[beam]];
  } else {
    int rank = 0;
    for (int j = 0; j < beam; ++j) rank += !keeps[j];
    target = slot[free_rank[rank]];
  }
  if (reports && tid == 0) p.slots_out[first + beam] = target;
  if (!copies) return;
  const int64_t at = blockIdx.z * p.layer_stride + blockIdx.y * kPiece;
  const uint4* src = reinterpret_cast<const uint4*>(p.pool + at + slot[parent[beam]] * p.slot_stride);
  uint4* dst = reinterpret_cast<uint4*>(p.pool + at + target * p.slot_stride);
  const int n = (int)(min(kPiece, p.row_bytes - blockIdx.y * kPiece) / 16);
  constexpr int kAhead = 8;
  for (int i = tid; i < n; i += kAhead * kReorderNT) {
    uint4 x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + j * kReorderNT < n) x[j] = __ldcs(src + i + j * kReorderNT);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + j * kReorderNT < n) __stcs(dst + i + j * kReorderNT, x[j]);
  }
}

}  // namespace

cudaError_t launch_beam_reorder(const ReorderParams& p, cudaStream_t stream) {
  const unsigned pieces = p.row_bytes > 0 ? (unsigned)((p.row_bytes - 1) / kPiece + 1) : 1u;
  beam_reorder_kernel<<<dim3(p.n * p.beams, pieces, p.layers > 0 ? p.layers : 1), kReorderNT, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
