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

constexpr int kRowNT = 256, kMergeNT = 256, kMostCandidates = 1024;

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
// groups; 0 where fewer groups have a number.  group[0..G) and *result = 0 are written and visible; NT / G threads share
// the comparisons of a group.
template <int NT, int G, typename U>
__device__ __forceinline__ U bound_of(const U* group, U* result, int best) {
  constexpr int kShare = NT / G;
  const int part = threadIdx.x % kShare;
  const U mine = group[threadIdx.x / kShare];
  int above = 0, same = 0;
#pragma unroll
  for (int i = part; i < G; i += kShare) {
    const U x = group[i];
    above += x > mine;
    same += x == mine;
  }
#pragma unroll
  for (int o = kShare / 2; o; o >>= 1) {
    above += shfl_xor(above, o);
    same += shfl_xor(same, o);
  }
  if (above < best && best <= above + same) *result = mine;  // (several threads write the same)
  __syncthreads();
  return *result;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two fp32 operations in one instruction (values as register pairs).
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Place in the slice of a thread's i-th value: VEC neighbours to a load.
template <int VEC>
__device__ __forceinline__ int place_of(int i) {
  return VEC * (threadIdx.x + i / VEC * kRowNT) + i % VEC;
}

// PER values a thread, in slices of up to 256 PER, four CTAs an SM so that the loads of one cover the work of the others
// (three: 122 us for 512 rows of 131,072 fp32 values, slices of half the size: 110; this: 83, 72 of it here).  Bound there by its
// instructions, about 24 a value, between barriers, at 55% of HBM; for few rows by the chain of load, maximum, bound and
// ranks of one slice.  VEC values to a load: 16 bytes of rows that are aligned to them (4: fp32, 8: bf16), else 1.
template <typename T, int PER, int VEC>
__global__ void __launch_bounds__(kRowNT, PER > 16 ? 4 : 6) beam_rows_kernel(BeamParams p, BeamWork w) {
  constexpr int kWarps = kRowNT / 32, kGroups = 2 * kMaxBeams;
  __shared__ __align__(16) uint32_t group[kGroups];
  __shared__ uint32_t bound;
  __shared__ uint64_t cand[kMostCandidates], w_best[kWarps];
  __shared__ uint32_t w_max[kWarps];
  __shared__ int w_coarse[kWarps], w_fine[kWarps], count, nan;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / w.slices, slice = blockIdx.x - row * w.slices;
  tc::grid_dep_launch();
  const int v0 = slice * w.slice_len, len = min(p.vocab - v0, w.slice_len);
  const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.stride + v0;
  float a[PER];
  if (VEC > 1 && len == PER * kRowNT) {  // a whole slice: all its loads are under way before the first is looked at
    uint4 u[PER / VEC];
#pragma unroll
    for (int i = 0; i < PER / VEC; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(x + place_of<VEC>(i * VEC)));
#pragma unroll
    for (int i = 0; i < PER / VEC; ++i) {
      const uint32_t y[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        a[i * VEC + e] = __uint_as_float(sizeof(T) == 4 ? y[e % 4] : e & 1 ? y[e / 2] & 0xffff0000u : y[e / 2] << 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) a[i] = place_of<VEC>(i) < len ? load_f(x + place_of<VEC>(i)) : -CUDART_INF_F;
  }
  float top = -CUDART_INF_F;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, a[i]);
  const uint32_t mine = order_of(top);
  // (up to 32 continuations are bounded by the maxima of 64 groups of 4 threads, more by those of 128 groups of 2)
  uint32_t g = max(mine, shfl_xor(mine, 1));
  const bool few = p.best <= kMaxBeams / 2;
  if (few) g = max(g, shfl_xor(g, 2));
  if ((lane & (few ? 3 : 1)) == 0) group[tid >> (few ? 2 : 1)] = g;
  g = __reduce_max_sync(0xffffffffu, mine);
  if (lane == 0) w_max[warp] = g;
  if (tid == 0) count = nan = bound = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) g = max(g, w_max[i]);
  const float m = g ? value_of(g) : -CUDART_INF_F;
  // The sum: each exponential's whole multiples of 2^-16 and what is left of it are added up apart.  A thread's additions
  // of multiples are exact, and so are a warp's sums as integers (of 2^-16: at most 32 PER 2^16; of 2^-33: as much).
  {
    static_assert(PER <= 32, "sums as 32-bit integers");
    const float ref = m == -CUDART_INF_F ? 0.f : m;
    const uint64_t mm = pair(-ref, -ref), log2e = pair(1.4426950408889634f, 1.4426950408889634f);
    const uint64_t up = pair(192.f, 192.f), down = pair(-192.f, -192.f);  // (in [2^7, 2^8): steps of 2^-16)
    const uint64_t minus = pair(-1.f, -1.f);
    uint64_t coarse = 0ull, fine = 0ull;
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      float t0, t1;
      unpair(mul2(add2(pair(a[i], a[i + 1]), mm), log2e), t0, t1);
      const uint64_t e = pair(exp2_fast(t0), exp2_fast(t1)), c = add2(add2(e, up), down);
      coarse = add2(coarse, c);
      fine = add2(fine, fma2(c, minus, e));
    }
    float c0, c1, f0, f1;
    unpair(coarse, c0, c1);
    unpair(fine, f0, f1);
    const float c = c0 + c1, f = f0 + f1;
    const bool bad = c != c;  // (a NaN among the values, or +inf - +inf)
    if (__any_sync(0xffffffffu, bad) && lane == 0) nan = 1;
    const int ci = __reduce_add_sync(0xffffffffu, bad ? 0 : (int)(c * 65536.f));
    const int fi = __reduce_add_sync(0xffffffffu, bad ? 0 : __float2int_rn(f * 8589934592.f));
    if (lane == 0) {
      w_coarse[warp] = ci;
      w_fine[warp] = fi;
    }
  }
  const uint32_t least = few ? bound_of<kRowNT, kGroups / 2>(group, &bound, p.best) : bound_of<kRowNT, kGroups>(group, &bound, p.best);
  if (tid == 0) {
    long long c = 0, f = 0;
    for (int i = 0; i < kWarps; ++i) {
      c += w_coarse[i];
      f += w_fine[i];
    }
    w.sum[blockIdx.x] = nan ? CUDART_NAN : (double)((c << 17) + f) * 0x1p-33;
    w.max[blockIdx.x] = m;
  }
  const float floor = least ? value_of(least) : -3.402823466e38f;
  if (top >= floor) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (a[i] >= floor) {
        const int v = place_of<VEC>(i);
        const uint64_t k = v < len ? key_of(a[i], v0 + v) : 0ull;
        if (k) {
          const int n = atomicAdd(&count, 1);
          if (n < kMostCandidates) cand[n] = k;
        }
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
        const int v = place_of<VEC>(i);
        const uint64_t c = v < len ? key_of(a[i], v0 + v) : 0ull;
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
  constexpr int kGroups = 64, kWarps = kMergeNT / 32;
  __shared__ double base[kMaxBeams];
  __shared__ unsigned long long group[kGroups], bound;
  __shared__ uint64_t total[kMostCandidates], w_total[kWarps];
  __shared__ int where[kMostCandidates], w_where[kWarps], count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, req = blockIdx.x;
  const int per_beam = w.slices * p.best, lists = p.beams * w.slices, n_all = lists * p.best;
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
  if (tid < kGroups) group[tid] = 0;
  if (tid == 0) count = bound = 0;
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
  // the bound from the lists' first entries, then every list from its first entry down to the bound
  for (int i = tid; i < lists; i += kMergeNT) atomicMax(&group[i % kGroups], (unsigned long long)total_of(i * p.best));
  __syncthreads();
  const uint64_t least = bound_of<kMergeNT, kGroups>(group, &bound, p.best);
  for (int i = tid; i < lists; i += kMergeNT)
    for (int e = 0; e < p.best; ++e) {
      const uint64_t t = total_of(i * p.best + e);
      if (!t || t < least) break;
      const int n = atomicAdd(&count, 1);
      if (n < kMostCandidates) {
        total[n] = t;
        where[n] = i * p.best + e;
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
// 8,192 (fewer lists and less fixed work for a value).
cudaError_t work_of(const BeamParams& p, BeamWork* w, int* per) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const long long rows = (long long)p.n * p.beams, small = (p.vocab - 1) / (8 * kRowNT) + 1;
  *per = rows * small <= 2 * sms ? 8 : 32;
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
  const bool wide = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.stride * (bf16 ? 2 : 4) % 16 == 0;
  auto rows = [&](auto kernel) { kernel<<<grid, kRowNT, 0, stream>>>(p, w); };
  if (bf16 && wide) rows(per == 8 ? beam_rows_kernel<__nv_bfloat16, 8, 8> : beam_rows_kernel<__nv_bfloat16, 32, 8>);
  else if (bf16) rows(per == 8 ? beam_rows_kernel<__nv_bfloat16, 8, 1> : beam_rows_kernel<__nv_bfloat16, 32, 1>);
  else if (wide) rows(per == 8 ? beam_rows_kernel<float, 8, 4> : beam_rows_kernel<float, 32, 4>);
  else rows(per == 8 ? beam_rows_kernel<float, 8, 1> : beam_rows_kernel<float, 32, 1>);
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
