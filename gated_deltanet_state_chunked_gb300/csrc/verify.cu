// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// Request i has `len` drafted tokens x_0.., the target's rows p_0..p_len and the draft's rows q_0..
//   draft j is accepted while u_j q_j(x_j) < p_j(x_j)      (exact: the product of two fp32 in fp64)
//   a = the number accepted before the first that is not; then one token is sampled by inverse CDF:
//   from W = max(p_a - q_a, 0) after a rejection (from p_a where W is all zero), from p_a otherwise:
//   the lowest index whose inclusive sum of W exceeds floor(u_w sum W).
// Probabilities enter the sums as whole multiples of 2^-44 (rounded down, clamped to [0, 1], NaN
// as 0): whole-number sums are the same in any order, so the token never depends on how the row is
// split over threads, and with at most 2^19 entries a sum stays below 2^63.
//
// Bound: reading one row of p and, after a rejection, one of q, once from HBM.
#include <cuda_bf16.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int NT = 1024, NWARP = NT / 32;
typedef unsigned long long u64;

__device__ __forceinline__ float prob(const float* p) { return *p; }
__device__ __forceinline__ float prob(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// floor(clamp(p, 0, 1) 2^44); NaN gives 0.
__device__ __forceinline__ u64 fixed44(float p) {
  const float c = p > 0.f ? (p < 1.f ? p : 1.f) : 0.f;
  return __float2ull_rz(c * 17592186044416.f);  // scaling by a power of two is exact
}

__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename Tp>
__global__ void __launch_bounds__(NT) verify_kernel(const VerifyParams p) {
  __shared__ int s_accept;
  __shared__ u64 s_rest[NWARP], s_last[NWARP];
  const int i = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = p.draft_lens ? p.draft_lens[i] : p.n_draft;
  if (len < 0) return;  // padding
  if (len > p.n_draft) {
    if (tid == 0) atomicExch(p.status, GDN_ERR_SHAPE);
    return;
  }
  const Tp* target = static_cast<const Tp*>(p.target);
  const Tp* draft = static_cast<const Tp*>(p.draft);
  const size_t trow = (size_t)i * (p.n_draft + 1), drow = (size_t)i * p.n_draft;
  if (warp == 0) {
    int a = len;
    for (int j0 = 0; j0 < len; j0 += 32) {
      const int j = j0 + lane;
      bool ok = true;
      if (j < len) {
        const int x = p.drafted[drow + j];
        ok = x >= 0 && x < p.vocab;
        if (ok) {
          const double pt = prob(target + (trow + j) * p.target_stride + x);
          const double pd = draft ? prob(draft + (drow + j) * p.draft_stride + x) : 1.0;
          ok = (double)p.uniforms[trow + j] * pd < pt;
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !ok);
      if (no) {
        a = j0 + __ffs(no) - 1;
        break;
      }
    }
    if (lane == 0) s_accept = a;
  }
  __syncthreads();
  const int a = s_accept;
  const bool rejected = a < len;
  const Tp* prow = target + (trow + a) * p.target_stride;
  const Tp* qrow = draft + (drow + a) * p.draft_stride;  // read only after a rejection with draft rows
  const int x_a = rejected ? p.drafted[drow + a] : -1;
  if (rejected && (x_a < 0 || x_a >= p.vocab) && tid == 0) atomicExch(p.status, GDN_ERR_SHAPE);
  const bool minus = rejected && draft;
  auto weight = [&](int v, u64& last) {
    last = fixed44(prob(prow + v));
    if (!rejected) return last;
    const u64 q = minus ? fixed44(prob(qrow + v)) : (v == x_a && !draft ? ~0ull : 0ull);
    return last > q ? last - q : 0ull;
  };
  // Each warp sums a range of the row of its own; then the warp that the sampled place falls into
  // walks its range again.
  const int per = ((p.vocab + NWARP - 1) / NWARP + 31) / 32 * 32;
  const int lo = min(warp * per, p.vocab), hi = min(lo + per, p.vocab);
  u64 rest = 0, last = 0;
  for (int v = lo + lane; v < hi; v += 32) {
    u64 l;
    rest += weight(v, l);
    last += l;
  }
  rest = warp_sum(rest);
  last = warp_sum(last);
  if (lane == 0) {
    s_rest[warp] = rest;
    s_last[warp] = last;
  }
  __syncthreads();
  u64 total_rest = 0, total_last = 0;
#pragma unroll 8
  for (int w = 0; w < NWARP; ++w) {
    total_rest += s_rest[w];
    total_last += s_last[w];
  }
  const bool use_rest = total_rest > 0;
  const u64 total = use_rest ? total_rest : total_last;
  int32_t* out = p.tokens + trow;
  if (total == 0) {  // nothing to sample from
    if (tid == 0) out[a] = -1;
  } else {
    const double r = floor((double)p.uniforms[trow + p.n_draft] * (double)total);
    // (r below 0 or NaN: the first place; r past the sum: the last)
    u64 place = r > 0.0 ? (r < 9.2e18 ? (u64)r : total - 1) : 0;
    place = place < total ? place : total - 1;
    u64 before = 0;
    for (int w = 0; w < warp; ++w) before += use_rest ? s_rest[w] : s_last[w];
    const u64 mine = use_rest ? s_rest[warp] : s_last[warp];
    if (place >= before && place - before < mine) {
      for (int v0 = lo; v0 < hi; v0 += 32) {
        const int v = v0 + lane;
        u64 l = 0, w = 0;
        if (v < hi) {
          w = weight(v, l);
          if (!use_rest) w = l;
        }
        u64 incl = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
        const unsigned over = __ballot_sync(0xffffffffu, before + incl > place);
        if (over) {
          if (lane == 0) out[a] = v0 + __ffs(over) - 1;
          break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
  }
  for (int j = tid; j <= p.n_draft; j += NT)
    if (j != a) out[j] = j < a ? p.drafted[drow + j] : -1;
  if (tid == 0) p.counts[i] = a + 1;
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, int bf16, cudaStream_t stream) {
  if (bf16) verify_kernel<__nv_bfloat16><<<p.n, NT, 0, stream>>>(p);
  else verify_kernel<float><<<p.n, NT, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
