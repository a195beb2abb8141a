// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// Request i has `len` drafted tokens x_0.., the target's rows p_0..p_len and the draft's rows q_0..
//   draft j is accepted while u_j q_j(x_j) < p_j(x_j)      (exact: the product of two fp32 in fp64)
//   a = the number accepted before the first that is not; then one token is sampled by inverse CDF:
//   from W = max(p_a - q_a, 0) after a rejection (from p_a where W is all zero), from p_a otherwise:
//   the lowest index whose inclusive sum of W exceeds floor(u_w sum W).
// Probabilities enter the sums as whole multiples of 2^-44 (rounded down, clamped to [0, 1], NaN
// as 0): whole-number sums are the same in any order, so the token never depends on how the row is
// split over threads, and with at most 2^19 entries a sum is at most 2^63, in unsigned 64 bits.
//
// A cluster of CTAs shares a request: each warp sums a range of the row of its own, the CTAs tell each
// other their totals through distributed shared memory, the warps of the one CTA whose part of the row
// holds the sampled place share the range that holds it, and one of them walks what is left of it.
//
// Bound: reading one row of p and, after a rejection, one of q, from HBM (128 requests over 131,072
// entries: 31 us, 18 us of reading), with the chain of dependent reads around it (drafts, their
// probabilities, the row, the walk: 6 us of one request over 32,000 entries).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <type_traits>
#include <utility>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
typedef unsigned long long u64;

// Four consecutive entries: in one load (aligned to their size), or the first `n` one by one (others 0).
__device__ __forceinline__ float4 load4(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float prob(const float* p) { return *p; }
__device__ __forceinline__ float prob(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <typename Tp>
__device__ __forceinline__ float4 load_some(const Tp* p, int n) {
  return make_float4(n > 0 ? prob(p) : 0.f, n > 1 ? prob(p + 1) : 0.f, n > 2 ? prob(p + 2) : 0.f, n > 3 ? prob(p + 3) : 0.f);
}

// F = floor(clamp(p, 0, 1) 2^44), NaN as 0, in two 22-bit halves: hi = floor(p 2^22), lo = floor of
// what is left times 2^22.  Adding 2^23 with rounding down leaves the floor in the mantissa; the halves
// keep the bits of 2^23 as a bias, which cancels in differences.  (A conversion to 64 bits does it in
// one instruction, at two a clock and SM: 85 us for 128 requests over 131,072 entries.)
struct Fixed {
  int hi, lo;
};
constexpr int kBias = 0x4b000000;  // the bits of 2^23
__device__ __forceinline__ Fixed fixed44(float p) {  // p in [0, 1]
  const float a = __fmaf_rd(p, 4194304.f, 8388608.f);
  const float rest = fmaf(p, 4194304.f, 8388608.f - a);  // exact: below 1, with p's last bit
  return {__float_as_int(a), __float_as_int(__fmaf_rd(rest, 4194304.f, 8388608.f))};
}
// Adds the halves of max(F(p) - F(q), 0) (each may be negative) to hi and lo: F is monotone, so the
// difference is positive or zero exactly where p > q or F(p) = F(q).
template <bool MINUS>
__device__ __forceinline__ void add_weight(float p, float q, int& hi, int& lo) {
  p = __saturatef(p);  // (NaN: 0)
  const Fixed x = fixed44(p);
  if (!MINUS) {
    hi += x.hi - kBias;
    lo += x.lo - kBias;
    return;
  }
  q = __saturatef(q);
  const Fixed y = fixed44(q);
  if (p > q) {
    hi += x.hi - y.hi;
    lo += x.lo - y.lo;
  }
}
__device__ __forceinline__ u64 joined(int hi, int lo) { return (u64)(((long long)hi << 22) + lo); }

__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// NT threads a CTA, MINB CTAs an SM, UNROLL groups of four entries a lane in flight.
template <typename Tp, int NT, int MINB, int UNROLL>
__global__ void __launch_bounds__(NT, MINB) verify_kernel(const VerifyParams p) {
  constexpr int NWARP = NT / 32;
  __shared__ int s_accept;
  __shared__ u64 s_warp[NWARP], s_sub[NWARP];
  __shared__ u64 s_cta[2][kMaxCluster];  // every CTA's total, of the weights, then (they are zero) of p alone
  const cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int i = blockIdx.x / ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Tp* target = static_cast<const Tp*>(p.target);
  const Tp* draft = static_cast<const Tp*>(p.draft);
  const size_t trow = (size_t)i * (p.n_draft + 1), drow = (size_t)i * p.n_draft;
  // (independent reads first: the length, the first drafts and the random numbers are one latency)
  const int len = p.draft_lens ? p.draft_lens[i] : p.n_draft;
  const float u_last = p.uniforms[trow + p.n_draft];
  int x0 = -1;
  float u0 = 0.f;
  if (warp == 0 && lane < p.n_draft) {
    x0 = p.drafted[drow + lane];
    u0 = p.uniforms[trow + lane];
  }
  if (len < 0) return;  // padding
  if (len > p.n_draft) {
    if (tid == 0) atomicExch(p.status, GDN_ERR_SHAPE);
    return;
  }
  auto begun = cluster.barrier_arrive();  // (waited for before the first write to another CTA's memory)
  if (warp == 0) {
    int a = len;
    for (int j0 = 0; j0 < len; j0 += 32) {
      const int j = j0 + lane;
      bool ok = true;
      if (j < len) {
        const int x = j0 == 0 ? x0 : p.drafted[drow + j];
        const float u = j0 == 0 ? u0 : p.uniforms[trow + j];
        ok = x >= 0 && x < p.vocab;
        if (ok) {
          const double pt = prob(target + (trow + j) * p.target_stride + x);
          const double pd = draft ? prob(draft + (drow + j) * p.draft_stride + x) : 1.0;
          ok = (double)u * pd < pt;
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
  const int x_a = rejected ? p.drafted[drow + a] : -1;
  if (rejected && (x_a < 0 || x_a >= p.vocab) && tid == 0 && rank == 0) atomicExch(p.status, GDN_ERR_SHAPE);
  // What is taken from p: the draft's row, or all of the rejected token.
  const Tp* qrow = rejected && draft ? draft + (drow + a) * p.draft_stride : nullptr;
  const int without = rejected && !draft ? x_a : -1;
  const bool vec = (reinterpret_cast<uintptr_t>(prow) | (qrow ? reinterpret_cast<uintptr_t>(qrow) : 0)) %
                       (4 * sizeof(Tp)) == 0;
  // Ranges of whole groups of 128 entries (four a lane), warp by warp, CTA by CTA.
  const int per = ((p.vocab + ctas * NWARP - 1) / (ctas * NWARP) + 127) / 128 * 128;
  int lo = min((rank * NWARP + warp) * per, p.vocab), hi = min(lo + per, p.vocab);
  // Halves of the weights of entries [v, v + 4) of the range, one after another.
  auto weights = [&](bool minus, int v, int (&wh)[4], int (&wl)[4]) {
    const bool whole = vec && v + 4 <= hi;
    const float4 t = whole ? load4(prow + v) : load_some(prow + v, hi - v);
    float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
    if (minus && qrow) d = whole ? load4(qrow + v) : load_some(qrow + v, hi - v);
    const float* tf = &t.x;
    const float* df = &d.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      wh[e] = wl[e] = 0;
      add_weight<true>(tf[e], df[e], wh[e], wl[e]);
    }
  };
  // Sums of the halves over this lane's entries (at most 256 of them: below 2^30).
  auto sums = [&](auto with_q, int& sh, int& sl) {
    constexpr bool Q = decltype(with_q)::value;
    const int whole = vec ? lo + (hi - lo) / 128 * 128 : lo;
#pragma unroll UNROLL
    for (int v = lo + 4 * lane; v < whole; v += 128) {
      const float4 t = load4(prow + v);
      const float4 d = Q ? load4(qrow + v) : make_float4(0.f, 0.f, 0.f, 0.f);
      add_weight<Q>(t.x, d.x, sh, sl);
      add_weight<Q>(t.y, d.y, sh, sl);
      add_weight<Q>(t.z, d.z, sh, sl);
      add_weight<Q>(t.w, d.w, sh, sl);
    }
    // (what is left of the range, or all of it when the rows are not aligned)
#pragma unroll 4
    for (int v = whole + lane; v < hi; v += 32) add_weight<Q>(prob(prow + v), Q ? prob(qrow + v) : 0.f, sh, sl);
  };
  bool minus = rejected;  // false: the weights are p's
  bool found = false;     // [lo, hi) is this warp's share of the range that holds the sampled place
  u64 place = 0;          // from the sum before that range
  const bool one_group = per == 128;
  for (int pass = 0;; ++pass) {
    int sh = 0, sl = 0;
    if (found && one_group) {}  // (what one step walks is not summed again)
    else if (minus && qrow) sums(std::true_type{}, sh, sl);
    else sums(std::false_type{}, sh, sl);
    if (minus && without >= lo && without < hi && lane == 0) {
      int wh = 0, wl = 0;
      add_weight<false>(prob(prow + without), 0.f, wh, wl);
      sh -= wh;
      sl -= wl;
    }
    const u64 sum = warp_sum(joined(sh, sl));
    if (found) {
      u64 before = 0;
      if (!one_group) {
        if (lane == 0) s_sub[warp] = sum;
        __syncthreads();
        for (int w = 0; w < warp; ++w) before += s_sub[w];
        if (place < before || place - before >= sum) return;
      }
      for (int v0 = lo; v0 < hi; v0 += 128) {
        int wh[4], wl[4];
        u64 w[4], incl = 0;
        weights(minus, v0 + 4 * lane, wh, wl);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = minus && v0 + 4 * lane + e == without ? 0ull : joined(wh[e], wl[e]);
          incl += w[e];
        }
        const u64 own = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
        const unsigned over = __ballot_sync(0xffffffffu, before + incl > place);
        if (over) {
          if (lane == __ffs(over) - 1) {
            const u64 s0 = before + incl - own + w[0], s1 = s0 + w[1], s2 = s1 + w[2];
            p.tokens[trow + a] = v0 + 4 * lane + (s0 > place ? 0 : s1 > place ? 1 : s2 > place ? 2 : 3);
          }
          return;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
      return;
    }
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    if (pass == 0) cluster.barrier_wait(std::move(begun));  // every CTA of the cluster runs
    if (tid < ctas) {
      u64 cta = 0;
#pragma unroll
      for (int w = 0; w < NWARP; ++w) cta += s_warp[w];
      cluster.map_shared_rank(&s_cta[pass][0], tid)[rank] = cta;
    }
    cluster.sync();
    u64 total = 0, before = 0;  // before: this CTA's part of the row
    for (int r = 0; r < ctas; ++r) {
      if (r == rank) before = total;
      total += s_cta[pass][r];
    }
    if (total == 0 && minus) {
      minus = false;  // nothing is left of p: it is sampled itself
      continue;
    }
    if (rank == 0) {
      int32_t* out = p.tokens + trow;
      for (int j = tid; j <= p.n_draft; j += NT)
        if (j != a || total == 0) out[j] = j < a ? p.drafted[drow + j] : -1;
      if (tid == 0) p.counts[i] = a + 1;
    }
    if (total == 0) return;
    const double r = floor((double)u_last * (double)total);
    // (r below 0 or NaN: the first place; r past the sum: the last)
    place = r > 0.0 ? (r < (double)total ? (u64)r : total - 1) : 0;
    place = place < total ? place : total - 1;  // ((double)total may be rounded up)
    if (place < before || place - before >= s_cta[pass][rank]) return;
    place -= before;
    int w = 0;
    while (place >= s_warp[w]) place -= s_warp[w++];
    found = true;
    if (one_group) {
      if (w != warp) return;
      continue;
    }
    // The warps share that range, in whole groups of 128 entries.
    const int from = (rank * NWARP + w) * per, to = min(from + per, p.vocab);
    const int share = (per / 128 + NWARP - 1) / NWARP * 128;
    lo = min(from + warp * share, to);
    hi = min(lo + share, to);
  }
}

template <typename Tp, int NT, int MINB, int UNROLL>
cudaError_t launch(const VerifyParams& p, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.n * ctas));
  cfg.blockDim = dim3(NT);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<Tp, NT, MINB, UNROLL>, p);
}

// CTAs per request: up to a portable cluster, while each gets 4096 entries.  Few requests take CTAs of
// 512 threads, at most two an SM: a cluster's CTAs are placed as densely as they fit, and smaller ones
// leave most SMs idle (16 requests over 131,072 entries: 11 us; 15 us against 24 us before the warps
// shared the last range).  With more CTAs than that places, small ones, eight an SM, start in one wave
// (128 requests: 31 us; 39 us against 49 us).
template <typename Tp>
cudaError_t launch_type(const VerifyParams& p, cudaStream_t stream) {
  constexpr int kTwoPerSm = 304;
  int ctas = 1;
  while (ctas < kMaxCluster && ctas * 4096 < p.vocab) ctas *= 2;
  if ((long long)p.n * ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  return p.n * ctas <= kTwoPerSm ? launch<Tp, 512, 2, 4>(p, ctas, stream) : launch<Tp, 256, 8, 2>(p, ctas, stream);
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, int bf16, cudaStream_t stream) {
  return bf16 ? launch_type<__nv_bfloat16>(p, stream) : launch_type<float>(p, stream);
}

}  // namespace gdn
