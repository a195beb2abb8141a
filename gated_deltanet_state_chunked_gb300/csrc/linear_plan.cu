// Planning of gdn_linear_attn: the work list, the entering states of cut sequences, and the order of
// launches (see linear_work.cuh).
#include <algorithm>
#include <atomic>
#include <climits>

#include "linear_work.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

// The plan of a call with several sequences, one CTA: `units` entries, the segments of every sequence
// with a valid range (longest first while they are at most kSortMost, else in order), then -1; `cut`
// entries of the segments of cut sequences alone; `cuts` entries of the cut sequences.  A range
// [cu[i], cu[i+1]) counts when 0 <= cu[i] <= cu[i+1] <= total_tokens and no earlier offset is above
// cu[i]; others are reported.  An empty sequence is one segment of no tokens.
constexpr int kPlanNT = 1024, kSortMost = 1024;
__global__ void __launch_bounds__(kPlanNT) linear_plan_kernel(const int32_t* cu, int n_seqs, int total, int seg_tokens,
                                                              Segment* list, int units, Segment* cut_list, int cut_units,
                                                              CutSeq* cuts, int n_cuts, int* status) {
  __shared__ int w_max[32], w_units[32], w_cut[32], w_cuts[32];
  __shared__ int key[kSortMost];
  tc::grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < units; i += kPlanNT) list[i].seq = -1;
  for (int i = tid; i < cut_units; i += kPlanNT) cut_list[i].seq = -1;
  for (int i = tid; i < n_cuts; i += kPlanNT) cuts[i].seq = -1;
  const bool sort = units <= kSortMost;
  if (sort)
    for (int i = tid; i < units; i += kPlanNT) key[i] = -1;
  int c_max = INT_MIN, c_units = 0, c_cut = 0, c_cuts = 0;
  __syncthreads();
  for (int base = 0; base < n_seqs; base += kPlanNT) {
    const int i = base + tid;
    int a = 0, b = INT_MIN, top = INT_MIN;
    if (i < n_seqs) {
      a = cu[i];
      b = cu[i + 1];
      top = max(a, b);
    }
    int incl = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl = max(incl, x);
    }
    int before = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) before = INT_MIN;
    if (lane == 31) w_max[warp] = incl;
    __syncthreads();
    int all = c_max;
    before = max(before, c_max);
    for (int w = 0; w < kPlanNT / 32; ++w) {
      if (w < warp) before = max(before, w_max[w]);
      all = max(all, w_max[w]);
    }
    const bool ok = i < n_seqs && a >= 0 && a >= before && b >= a && b <= total;
    if (i < n_seqs && !ok) atomicExch(status, GDN_ERR_SHAPE);
    const int n = ok ? segments_of(b - a, seg_tokens) : 0;
    // inclusive sums of segments, segments of cut sequences, cut sequences
    int su = n, sc = n > 1 ? n : 0, sq = n > 1 ? 1 : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int xu = __shfl_up_sync(0xffffffffu, su, o), xc = __shfl_up_sync(0xffffffffu, sc, o),
                xq = __shfl_up_sync(0xffffffffu, sq, o);
      if (lane >= o) { su += xu; sc += xc; sq += xq; }
    }
    if (lane == 31) { w_units[warp] = su; w_cut[warp] = sc; w_cuts[warp] = sq; }
    __syncthreads();
    int bu = c_units, bc = c_cut, bq = c_cuts;
    for (int w = 0; w < kPlanNT / 32; ++w) {
      if (w < warp) { bu += w_units[w]; bc += w_cut[w]; bq += w_cuts[w]; }
      c_units += w_units[w];
      c_cut += w_cut[w];
      c_cuts += w_cuts[w];
    }
    c_max = all;
    bu += su - n;
    bc += sc - (n > 1 ? n : 0);
    bq += sq - (n > 1 ? 1 : 0);
    for (int j = 0; j < n; ++j) {
      Segment s = {};
      s.seq = i; s.seg = j; s.n_seg = n; s.t_begin = a + j * (n > 1 ? seg_tokens : 0);
      s.len = min(seg_tokens, b - s.t_begin); s.local = n > 1 ? bc + j : 0;
      if (bu + j < units) {
        list[bu + j] = s;
        if (sort) key[bu + j] = s.len;
      }
      if (n > 1 && bc + j < cut_units) cut_list[bc + j] = s;
    }
    if (n > 1 && bq < n_cuts) cuts[bq] = CutSeq{i, n, bc, b - (a + (n - 1) * seg_tokens)};
    __syncthreads();
  }
  if (!sort) return;
  const int u = tid;
  Segment s = {};
  int rank = 0;
  const bool have = u < units && key[u] >= 0;
  if (have) {
    s = list[u];
    for (int j = 0; j < units; ++j) rank += key[j] > s.len || (key[j] == s.len && j < u);
  }
  __syncthreads();
  if (have) list[rank] = s;
}

// The entering states of a cut sequence's segments, in place of the segments' own states, and (FINAL)
// the state behind the last one.  Element by element: E <- lambda^seg E + local; the loads of eight
// segments are under way at once (they do not depend on E, but a store between them would hold them up).
constexpr int kCarryNT = 256, kAhead = 8;
template <bool FINAL>
__global__ void __launch_bounds__(kCarryNT) linear_carry_kernel(const LinearWork p) {
  const int h = blockIdx.x % p.h_v, i = blockIdx.x / p.h_v;
  tc::grid_dep_launch();
  tc::grid_dep_wait();  // the segments' own states
  CutSeq q = {};
  if (p.cuts) {
    q = p.cuts[i];
  } else {
    const Segment s = only_segment(p, 0);
    q.seq = s.seq;
    q.n_seg = s.n_seg;
    q.last_len = s.seq < 0 ? 0 : p.cu[1] - (p.cu[0] + (s.n_seg - 1) * p.seg_tokens);
  }
  if (q.seq < 0 || q.n_seg < 2) return;
  const float g = p.log_decay[h];
  const int dd = p.d_v * p.d_k;
  const int e = (blockIdx.y * kCarryNT + threadIdx.x) * 4;
  if (e >= dd) return;
  const size_t at = ((size_t)q.seq * p.h_v + h) * dd + e, stride = (size_t)p.h_v * dd;
  float4 E = p.S0 ? *reinterpret_cast<const float4*>(p.S0 + at) : make_float4(0.f, 0.f, 0.f, 0.f);
  const DecayStep step = decay_step(g, p.seg_tokens), last = decay_step(g, q.last_len);
  float* loc = p.local + ((size_t)q.local * p.h_v + h) * dd + e;
  const int n_read = FINAL ? q.n_seg : q.n_seg - 1;  // (the last segment's own state is needed behind it only)
  for (int j0 = 0; j0 < q.n_seg; j0 += kAhead) {
    float4 x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      x[j] = j0 + j < n_read ? *reinterpret_cast<const float4*>(loc + (size_t)(j0 + j) * stride)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (j0 + j >= q.n_seg) break;
      if (!FINAL) *reinterpret_cast<float4*>(loc + (size_t)(j0 + j) * stride) = E;
      const DecayStep f = j0 + j + 1 == q.n_seg ? last : step;
      E = make_float4(f(E.x, x[j].x), f(E.y, x[j].y), f(E.z, x[j].z), f(E.w, x[j].w));
    }
  }
  if (FINAL) *reinterpret_cast<float4*>(p.S_out + at) = E;
}

// Cutting costs a launch for the segments' own states and one for their entering states, about 10 us on
// the tensor cores and 5 us on the CUDA cores, and saves a chunk's time for each chunk that runs beside
// others: 3 us for 128 tokens on the tensor cores (1024 tokens, 32 heads: 29 us cut in four, 35 us whole;
// 256 tokens: 23 and 12 us), 9 to 20 us for 64 tokens on the CUDA cores, where a segment of one chunk
// pays (2 heads of 128, 128 tokens: 34 us cut in two, 44 us whole; 1024 tokens: 36 us, 63 us at segments
// of two chunks, 324 us whole).
constexpr int kChunkTc = 128, kChunkSimt = 64;  // segments are whole chunks
constexpr int kMinSegmentTc = 256, kMinTokensTc = 1024;

// SMs of the current device, looked up once.
cudaError_t device_sms(int* sms) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
  *sms = known[dev].load(std::memory_order_relaxed);
  if (*sms > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) known[dev].store(*sms, std::memory_order_relaxed);
  return e;
}

// Tokens per segment: one sequence's segments times the v-heads fill the GPU once.
int segment_tokens(int total_tokens, int h_v, int sms, bool tc) {
  if (total_tokens < (tc ? kMinTokensTc : 1)) return INT_MAX;
  const int parts = std::max(1, sms / h_v);
  const int chunk = tc ? kChunkTc : kChunkSimt;
  const long long seg = ((total_tokens - 1) / parts / chunk + 1LL) * chunk;
  return seg >= total_tokens ? INT_MAX : tc ? std::max((int)seg, kMinSegmentTc) : (int)seg;
}

// What a call keeps in its workspace: the plan's lists (none for one sequence), the cut segments' states.
struct Workspace {
  int seg, units, cut_units, cuts;
  size_t list, cut_list, cut_seqs, local, bytes;
};
Workspace workspace_of(const LinearParams& p, int sms, bool tc) {
  Workspace w = {};
  const int seg = segment_tokens(p.total_tokens, p.h_v, sms, tc);
  const bool cut = seg < p.total_tokens;
  w.seg = cut ? seg : INT_MAX;
  // sum of max(1, ceil(len / seg)) <= n + total / seg; a cut sequence is longer than seg
  w.cuts = cut ? std::min(p.n_seqs, p.total_tokens / seg) : 0;
  w.cut_units = cut ? w.cuts + p.total_tokens / seg : 0;
  w.units = p.n_seqs + (cut ? p.total_tokens / seg : 0);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  if (p.n_seqs > 1) {
    w.list = take(sizeof(Segment) * (size_t)w.units);
    w.cut_list = take(sizeof(Segment) * (size_t)w.cut_units);
    w.cut_seqs = take(sizeof(CutSeq) * (size_t)w.cuts);
  }
  w.local = take((size_t)w.cut_units * p.h_v * p.d_v * p.d_k * 4);
  w.bytes = at;
  return w;
}

}  // namespace

// bf16 inputs run on the tensor cores (a call of no tokens has nothing for them to do).
static bool on_tensor_cores(const LinearParams& p, int bf16) { return bf16 && p.total_tokens > 0; }

cudaError_t linear_workspace_bytes(const LinearParams& p, int bf16, size_t* bytes) {
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e == cudaSuccess) *bytes = workspace_of(p, sms, on_tensor_cores(p, bf16)).bytes;
  return e;
}

cudaError_t launch_linear(const LinearParams& lp, int bf16, void* workspace, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const bool tc = on_tensor_cores(lp, bf16);
  const Workspace w = workspace_of(lp, sms, tc);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const bool cut = w.cuts > 0, plan = lp.n_seqs > 1;
  LinearWork p{};
  p.q = lp.q; p.k = lp.k; p.v = lp.v; p.log_decay = lp.log_decay; p.cu = lp.cu; p.S0 = lp.S0;
  p.local = reinterpret_cast<float*>(ws + w.local); p.O = lp.O; p.S_out = lp.S_out; p.status = lp.status;
  p.n_seqs = lp.n_seqs; p.total_tokens = lp.total_tokens; p.h_k = lp.h_k; p.h_v = lp.h_v; p.d_k = lp.d_k; p.d_v = lp.d_v;
  p.seg_tokens = w.seg; p.cut_units = w.cut_units; p.scale = lp.scale;
  Segment* list = plan ? reinterpret_cast<Segment*>(ws + w.list) : nullptr;
  Segment* cut_list = plan ? reinterpret_cast<Segment*>(ws + w.cut_list) : nullptr;
  CutSeq* cuts = plan ? reinterpret_cast<CutSeq*>(ws + w.cut_seqs) : nullptr;
  if (plan) {
    linear_plan_kernel<<<1, kPlanNT, 0, stream>>>(lp.cu, lp.n_seqs, lp.total_tokens, w.seg, list, w.units, cut_list,
                                                  w.cut_units, cuts, w.cuts, lp.status);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  p.list = list;
  p.cuts = cuts;
  const auto items = tc ? launch_linear_tc_items : launch_linear_simt_items;
  if (!lp.write_O) {
    p.early = plan;
    e = items(p, false, w.units, stream);
  } else if (cut) {
    LinearWork own = p;
    own.list = cut_list;
    own.local_only = 1;
    own.early = plan;
    e = items(own, false, w.cut_units, stream);
  }
  if (e != cudaSuccess) return e;
  if (cut) {
    const dim3 grid((unsigned)(w.cuts * lp.h_v), (lp.d_v * lp.d_k / 4 + kCarryNT - 1) / kCarryNT);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kCarryNT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = lp.write_O ? cudaLaunchKernelEx(&cfg, linear_carry_kernel<false>, p)
                   : cudaLaunchKernelEx(&cfg, linear_carry_kernel<true>, p);
    if (e != cudaSuccess) return e;
  }
  if (!lp.write_O) return cudaSuccess;
  p.early = plan || cut;
  return items(p, true, w.units, stream);
}

}  // namespace gdn
