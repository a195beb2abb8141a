// gdn_beam_select: the best continuations over beams and vocabulary.
//
// total(b, v) = (score_b - lse_b) + x_bv, lse_b = log sum_v exp(x_bv), in two kernels.  beam_rows_kernel cuts every row
// of logits into slices, one CTA each, which holds its slice in registers (the row is read once): the slice's
// maximum, its sum of exponentials and its `best` largest values.  beam_merge_kernel, one CTA a request, joins the sums
// and picks among the slices' lists.  Totals are compared in fp64, and the sums behind lse_b carry about 30 bits, so that
// the order of two beams' totals does not hang on roundings.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "gdn_internal.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

constexpr int kRowNT = 512, kMergeNT = 256, kMostCandidates = 1024;

struct BeamWork {
  double* sum;    // [rows][slices]: sum of exp(x - max) of a slice
  float* max;     // [rows][slices]
  uint64_t* keys; // [rows][slices][best], largest first
  int slices, slice_len;
};

// Numbers as unsigned integers of the same order; 0 (below all of them) for -inf, what is masked, and NaN.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return x > -CUDART_INF_F ? ((u & 0x80000000u) ? ~u : u | 0x80000000u) : 0u;
}
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o); }
__device__ __forceinline__ uint64_t order_of(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return x > -CUDART_INF ? ((u >> 63) ? ~u : u | 0x8000000000000000ull) : 0ull;
}
__device__ __forceinline__ double value_of(uint64_t o) {
  return __longlong_as_double((long long)((o >> 63) ? o & 0x7fffffffffffffffull : ~o));
}
// A value and its place in the row, the lower index first among equals: one 64-bit key, 0 for what is no candidate.
__device__ __forceinline__ uint64_t key_of(float x, int v) {
  const uint32_t o = order_of(x);
  return o ? (uint64_t)o << 32 | (uint32_t)~v : 0ull;
}

__device__ __forceinline__ float load_f(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}

template <typename U>
__device__ __forceinline__ U shfl_xor(U x, int o) {
  return (U)__shfl_xor_sync(0xffffffffu, x, o);
}
__device__ __forceinline__ uint64_t shfl_xor(uint64_t x, int o) {
  return (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)x, o);
}

// A bound that `best` numbers of the CTA at least reach and few others do: the best-th largest of the maxima of G
// groups of threads; 0 where fewer groups have a number.  group[0..G) written by the caller.
template <int G, typename U>
__device__ __forceinline__ U bound_of(const U* group, U* result, int best) {
  if (threadIdx.x == 0) *result = 0;
  __syncthreads();
  if (threadIdx.x < G) {
    const U mine = group[threadIdx.x];
    int above = 0, same = 0;
#pragma unroll 16
    for (int i = 0; i < G; ++i) {
      const U x = group[i];
      above += x > mine;
      same += x == mine;
    }
    if (above < best && best <= above + same) *result = mine;  // (several threads write the same)
  }
  __syncthreads();
  return *result;
}

// PER values a thread, in slices of up to 512 PER.  Bound by HBM where there are many rows: 15 instructions a value beside
// its load; for few rows by the chain of loads, maximum, bound and ranks of one slice.
template <typename T, int PER>
__global__ void __launch_bounds__(kRowNT, 2) beam_rows_kernel(BeamParams p, BeamWork w) {
  constexpr int kGroups = kRowNT / 4, kWarps = kRowNT / 32;
  __shared__ __align__(16) uint32_t group[kGroups];
  __shared__ uint32_t bound;
  __shared__ uint64_t cand[kMostCandidates], w_best[kWarps];
  __shared__ float w_max[kWarps];
  __shared__ double w_sum[kWarps];
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / w.slices, slice = blockIdx.x - row * w.slices;
  tc::grid_dep_launch();
  const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
  const int v0 = slice * w.slice_len, v1 = min(p.vocab, v0 + w.slice_len);
  float a[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int v = v0 + tid + i * kRowNT;
    a[i] = v < v1 ? load_f(x + v) : -CUDART_INF_F;
  }
  float top = -CUDART_INF_F;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, a[i]);
  const uint32_t mine = order_of(top);
  uint32_t g = max(mine, shfl_xor(mine, 1));
  g = max(g, shfl_xor(g, 2));
  if ((lane & 3) == 0) group[tid >> 2] = g;
  float m = top;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, shfl_xor(m, o));
  if (lane == 0) w_max[warp] = m;
  if (tid == 0) count = 0;
  __syncthreads();
  m = w_max[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) m = fmaxf(m, w_max[i]);
  // The sum: each exponential's whole multiples of 2^-16 and what is left of it are added up apart, so that a thread's
  // additions lose nothing (the multiples' sum is exact), and the threads' sums in fp64.
  {
    const float ref = m == -CUDART_INF_F ? 0.f : m;
    float coarse = 0.f, fine = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float e = expf(a[i] - ref), c = (e + 192.f) - 192.f;  // (192 lies in [2^7, 2^8): steps of 2^-16)
      coarse += c;
      fine += e - c;
    }
    double s = (double)coarse + (double)fine;
#pragma unroll
    for (int o = 16; o; o >>= 1) s += shfl_xor(s, o);
    if (lane == 0) w_sum[warp] = s;
  }
  const uint32_t least = bound_of<kGroups>(group, &bound, p.best);
  if (tid == 0) {
    double s = 0.;
    for (int i = 0; i < kWarps; ++i) s += w_sum[i];
    w.sum[blockIdx.x] = s;
    w.max[blockIdx.x] = m;
  }
  if (mine >= least) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int v = v0 + tid + i * kRowNT;
      const uint64_t k = v < v1 ? key_of(a[i], v) : 0ull;
      if (k && (uint32_t)(k >> 32) >= least) {
        const int n = atomicAdd(&count, 1);
        if (n < kMostCandidates) cand[n] = k;
      }
    }
  }
  __syncthreads();
  const int n = count;
  uint64_t* out = w.keys + (size_t)blockIdx.x * p.best;
  if (n <= kMostCandidates) {  // ranks by counting: keys differ
    for (int i = tid; i < n; i += kRowNT) {
      const uint64_t k = cand[i];
      int above = 0;
      for (int j = 0; j < n; ++j) above += cand[j] > k;
      if (above < p.best) out[above] = k;
    }
    for (int i = n + tid; i < p.best; i += kRowNT) out[i] = 0;
  } else {  // many equal values, or large ones in few threads: the largest key below the last one, again and again
    uint64_t last = ~0ull;
    for (int r = 0; r < p.best; ++r) {
      uint64_t k = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int v = v0 + tid + i * kRowNT;
        const uint64_t c = v < v1 ? key_of(a[i], v) : 0ull;
        if (c < last && c > k) k = c;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) k = max(k, shfl_xor(k, o));
      if (lane == 0) w_best[warp] = k;
      __syncthreads();
      k = w_best[0];
      for (int i = 1; i < kWarps; ++i) k = max(k, w_best[i]);
      __syncthreads();
      if (tid == 0) out[r] = k;
      last = k;
    }
  }
}

// A request's candidates are its beams' slices' lists: candidate i is entry i % best of list i / best, a beam's lists side
// by side.  Of equal totals the lower beam stands first, and within a beam the larger key.
__global__ void __launch_bounds__(kMergeNT, 3) beam_merge_kernel(BeamParams p, BeamWork w) {
  constexpr int kGroups = kMergeNT / 4, kWarps = kMergeNT / 32;
  __shared__ double base[kMaxBeams];
  __shared__ uint64_t group[kGroups], bound, total[kMostCandidates], w_total[kWarps];
  __shared__ int where[kMostCandidates], w_where[kWarps], count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, req = blockIdx.x;
  const int per_beam = w.slices * p.best, n_all = p.beams * per_beam;
  tc::grid_dep_wait();
  const size_t first = (size_t)req * p.beams * w.slices;
  const uint64_t* keys = w.keys + first * p.best;
  for (int b = warp; b < p.beams; b += kWarps) {
    float m = -CUDART_INF_F;
    for (int i = lane; i < w.slices; i += 32) m = fmaxf(m, w.max[first + b * w.slices + i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, shfl_xor(m, o));
    double s = 0.;
    for (int i = lane; i < w.slices; i += 32) {
      const double part = w.sum[first + b * w.slices + i];
      const float mi = w.max[first + b * w.slices + i];
      if (part != 0.) s += mi == m ? part : part * exp((double)mi - (double)m);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += shfl_xor(s, o);
    if (lane == 0) base[b] = (double)p.scores[(size_t)req * p.beams + b] - ((double)m + log(s));
  }
  if (tid == 0) count = 0;
  __syncthreads();
  auto total_of = [&](int i) -> uint64_t {
    const uint64_t k = keys[i];
    return k ? order_of(base[i / per_beam] + (double)value_of((uint32_t)(k >> 32))) : 0ull;
  };
  auto ahead = [&](int i, int j) {  // of equal totals
    const int bi = i / per_beam, bj = j / per_beam;
    return bi != bj ? bi < bj : keys[i] > keys[j];
  };
  auto put = [&](int r, uint64_t t, int i) {
    const size_t out = (size_t)req * p.best + r;
    p.scores_out[out] = t ? (float)value_of(t) : -CUDART_INF_F;
    p.parents[out] = t ? i / per_beam : -1;
    p.tokens[out] = t ? (int)~(uint32_t)keys[i] : -1;
  };
  uint64_t top = 0;
  for (int i = tid; i < n_all; i += kMergeNT) top = max(top, total_of(i));
  uint64_t g = max(top, shfl_xor(top, 1));
  g = max(g, shfl_xor(g, 2));
  if ((lane & 3) == 0) group[tid >> 2] = g;
  const uint64_t least = bound_of<kGroups>(group, &bound, p.best);
  if (top >= least)
    for (int i = tid; i < n_all; i += kMergeNT) {
      const uint64_t t = total_of(i);
      if (t && t >= least) {
        const int n = atomicAdd(&count, 1);
        if (n < kMostCandidates) {
          total[n] = t;
          where[n] = i;
        }
      }
    }
  __syncthreads();
  const int n = count;
  if (n <= kMostCandidates) {
    for (int i = tid; i < n; i += kMergeNT) {
      const uint64_t t = total[i];
      const int at = where[i];
      int above = 0;
      for (int j = 0; j < n; ++j) above += total[j] > t || (total[j] == t && j != i && ahead(where[j], at));
      if (above < p.best) put(above, t, at);
    }
    for (int i = n + tid; i < p.best; i += kMergeNT) put(i, 0, 0);
  } else {
    uint64_t last = ~0ull;
    int last_at = 0;
    for (int r = 0; r < p.best; ++r) {
      uint64_t t = 0;
      int at = 0;
      for (int i = tid; i < n_all; i += kMergeNT) {
        const uint64_t c = total_of(i);
        if (!c || c > last || (c == last && r > 0 && (i == last_at || !ahead(last_at, i)))) continue;
        if (c > t || (c == t && ahead(i, at))) {
          t = c;
          at = i;
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const uint64_t ot = shfl_xor(t, o);
        const int oa = shfl_xor(at, o);
        if (ot > t || (ot == t && t && oa != at && ahead(oa, at))) {
          t = ot;
          at = oa;
        }
      }
      if (lane == 0) {
        w_total[warp] = t;
        w_where[warp] = at;
      }
      __syncthreads();
      t = w_total[0];
      at = w_where[0];
      for (int i = 1; i < kWarps; ++i)
        if (w_total[i] > t || (w_total[i] == t && t && w_where[i] != at && ahead(w_where[i], at))) {
          t = w_total[i];
          at = w_where[i];
        }
      __syncthreads();
      if (tid == 0) put(r, t, at);
      last = t;
      last_at = at;
    }
  }
}

// Slices of 2,048 values while all of them together are at most two CTAs an SM (a row's latency counts), else of
// 16,384 (fewer lists and fixed work for each value).
cudaError_t work_of(const BeamParams& p, BeamWork* w, int* per) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const long long rows = (long long)p.n * p.beams, small = (p.vocab - 1) / (4 * kRowNT) + 1;
  *per = rows * small <= 2 * sms ? 4 : 32;
  w->slice_len = *per * kRowNT;
  w->slices = (p.vocab - 1) / w->slice_len + 1;
  return e;
}

}  // namespace

cudaError_t beam_workspace_bytes(const BeamParams& p, size_t* bytes) {
  BeamWork w;
  int per;
  const cudaError_t e = work_of(p, &w, &per);
  *bytes = (size_t)p.n * p.beams * w.slices * (sizeof(double) + sizeof(uint64_t) * p.best + sizeof(float));
  return e;
}

cudaError_t launch_beam_select(const BeamParams& p, int bf16, void* workspace, cudaStream_t stream) {
  BeamWork w;
  int per;
  cudaError_t e = work_of(p, &w, &per);
  if (e != cudaSuccess) return e;
  const size_t lists = (size_t)p.n * p.beams * w.slices;
  w.sum = static_cast<double*>(workspace);
  w.keys = reinterpret_cast<uint64_t*>(w.sum + lists);
  w.max = reinterpret_cast<float*>(w.keys + lists * p.best);
  const unsigned grid = (unsigned)lists;
  if (bf16) {
    if (per == 4) beam_rows_kernel<__nv_bfloat16, 4><<<grid, kRowNT, 0, stream>>>(p, w);
    else beam_rows_kernel<__nv_bfloat16, 32><<<grid, kRowNT, 0, stream>>>(p, w);
  } else {
    if (per == 4) beam_rows_kernel<float, 4><<<grid, kRowNT, 0, stream>>>(p, w);
    else beam_rows_kernel<float, 32><<<grid, kRowNT, 0, stream>>>(p, w);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n);
  cfg.blockDim = dim3(kMergeNT);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_merge_kernel, p, w);
}

}  // namespace gdn
