// Recurrent form on a pool of states: one token, or a short window of tokens, per request.
//
// Method: "Tail-Replay: Escaping the Curse of Linear Attention in Prefix Caching for Hybrid LLMs",
// section 2 Eq. (1), token by token; per v-head, with the state S (d_v x d_k) of the request:
//   delta rule     S <- alpha S (I - beta k k^T) + beta v k^T
//   scalar decay   S <- alpha S + beta v k^T
//   head decay     S <- lambda_h S + v k^T
// and the readout o = S (scale q) with the updated state.  A window of up to W tokens is unrolled on
// the state before it, so that a state is read, and written, once and every product with it stands
// by itself: with a_t = S k_t, b_t = S q_t, R_it = alpha_{i+1} .. alpha_t and c_t = alpha_1 .. alpha_t
//   d_t = beta_t (v_t - c_t a_t - sum_{i<t} R_it (k_i.k_t) d_i)        (delta rule; else beta_t v_t)
//   o_t = c_t b_t + sum_{i<=t} R_it (k_i.q_t) d_i
//   S  <- c_w S + sum_i R_iw d_i k_i^T
// row by row of S: the products k_i.k_t, k_i.q_t are computed once per CTA, and a row's a_t, b_t are
// reduced over the lanes that share it.  Longer windows go W tokens at a time, the state in registers.
//
// Layout: eight lanes share a row, lane l holding columns 4 (l & 7) + 32 j + [0, 4), so a warp's load
// covers four rows in whole 128-byte lines.
//
// Bound: HBM, 8 d_k d_v bytes per (request, v-head), for single tokens.  Windows are bound by their
// instructions (64 windows of 5 tokens, 32 heads of 128: 1290 a warp, 70 us with outputs against 20 us
// of reading, 65 us committed against 38 us of traffic): two products of the whole state for each
// token.  Measured and left: the products k_i.k_t from keys held in registers (they spill: 82 us),
// keys and queries fetched before the state (77 us).
#include <cuda_bf16.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
// Two fp32 fused multiply-adds in one instruction (values as register pairs).
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float pair_sum(uint64_t x) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
  return a + b;
}
__device__ __forceinline__ float4 scale4(float4 a, float s) { return make_float4(a.x * s, a.y * s, a.z * s, a.w * s); }
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A window's products of keys and queries are worth sharing over a whole state: sixteen warps for
// windows, eight for single tokens.  Either way 32 warps per SM at 64 registers a thread: what these
// kernels need most is loads in flight (256 requests of 32 heads, one token: 165 to 171 us, 95% of the
// rate of a copy, against 176 us at 24 warps and 216 us at 16).
__host__ __device__ constexpr int threads_of(int W) { return W == 1 ? 256 : 512; }

// J: column groups of 32 (d_k at most 32 J); W: tokens unrolled at once; RG: groups of four rows per
// warp (1 or 2).  DELTA: the delta rule.
template <typename Tin, int J, int W, int RG, bool DELTA>
__global__ void __launch_bounds__(threads_of(W), 1024 / threads_of(W)) decode_kernel(const DecodeParams p) {
  constexpr int NT = threads_of(W), NW = NT / 32;
  static_assert(W <= NW && (RG == 1 || RG == 2), "one warp prepares one token; two rows share eight lanes");
  __shared__ __align__(16) float ks[W][kMaxHead], qs[W][kMaxHead];  // normalised, queries times scale
  __shared__ float alpha[W], beta[W];
  __shared__ __align__(16) float kk[W][W], kq[W][W];  // [t][i]: k_i.k_t and k_i.q_t times R_it
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i = blockIdx.x, h = blockIdx.y;
  const int slot = p.slots ? p.slots[i] : i;
  if (slot < 0) return;  // padding
  const int cnt = p.counts ? p.counts[i] : p.window;
  if (slot >= p.n_slots || cnt < 0 || cnt > p.window) {
    if (tid == 0) atomicExch(p.status, GDN_ERR_SHAPE);
    return;
  }
  if (cnt == 0) return;
  const int hk = h / (p.h_v / p.h_k);
  const int col0 = 4 * (lane & 7);
  const int row0 = blockIdx.z * (NW * 4 * RG) + warp * (4 * RG) + (lane >> 3);
  float* Sb = p.S + ((size_t)slot * p.h_v + h) * p.d_v * p.d_k;
  float4 s[RG][J];
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = row0 + 4 * r, col = col0 + 32 * j;
      s[r][j] = (row < p.d_v && col < p.d_k) ? __ldcs(reinterpret_cast<const float4*>(Sb + (size_t)row * p.d_k + col))
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  // Two requests on one slot would race on its state: the first that updates it has it, the others
  // are skipped and reported.  (Checked while the state's loads are in flight.)
  if (p.slots && !p.keep) {
    int dup = 0;
    for (int j = tid; j < i; j += NT)
      dup |= p.slots[j] == slot && (!p.counts || (p.counts[j] > 0 && p.counts[j] <= p.window));
    if (__syncthreads_or(dup)) {
      if (tid == 0) atomicExch(p.status, GDN_ERR_SHAPE);
      return;
    }
  }
  const bool want_o = !p.state_only;
  const Tin* qp = static_cast<const Tin*>(p.q);
  const Tin* kp = static_cast<const Tin*>(p.k);
  const Tin* vp = static_cast<const Tin*>(p.v);
  Tin* op = static_cast<Tin*>(p.O);
  // the row whose sums this lane ends up with
  const int my_r = RG == 2 ? (lane >> 2) & 1 : 0;
  const int my_row = row0 + 4 * my_r;
  // products of this lane group's rows with x (this lane's columns), summed over a row's eight lanes;
  // with two rows, half of the lanes end up with each
  auto row_sum = [&](const float* x) {
    uint64_t y2[RG];
#pragma unroll
    for (int r = 0; r < RG; ++r) y2[r] = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(x + 32 * j);
#pragma unroll
      for (int r = 0; r < RG; ++r)
        y2[r] = fma2(pair(s[r][j].z, s[r][j].w), u.y, fma2(pair(s[r][j].x, s[r][j].y), u.x, y2[r]));
    }
    float y[RG];
#pragma unroll
    for (int r = 0; r < RG; ++r) y[r] = pair_sum(y2[r]);
    float z = my_r ? y[RG - 1] : y[0];
    z += __shfl_xor_sync(0xffffffffu, RG == 2 && !my_r ? y[RG - 1] : y[0], 4);
    z += __shfl_xor_sync(0xffffffffu, z, 2);
    return z + __shfl_xor_sync(0xffffffffu, z, 1);
  };
  for (int t0 = 0; t0 < cnt; t0 += W) {
    const int m = min(W, cnt - t0);
    const size_t tok0 = (size_t)i * p.window + t0;
    float v[W];
#pragma unroll
    for (int t = 0; t < W; ++t)
      v[t] = t < m && my_row < p.d_v ? load1(vp + ((tok0 + t) * p.h_v + h) * p.d_v + my_row) : 0.f;
    if (t0 > 0) __syncthreads();  // the tables of the tokens before are read
    if (warp < m) {
      const size_t tok = tok0 + warp;
      const bool in = 4 * lane < p.d_k;
      float4 k = make_float4(0.f, 0.f, 0.f, 0.f), q = k;
      if (in) {
        k = load4(kp + (tok * p.h_k + hk) * p.d_k + 4 * lane);
        if (want_o) q = load4(qp + (tok * p.h_k + hk) * p.d_k + 4 * lane);
      }
      if (lane == 0) {
        alpha[warp] = expf(p.family == kHeadDecay ? p.g[h] : p.g[tok * p.h_v + h]);
        beta[warp] = p.family == kHeadDecay ? 1.f : p.beta[tok * p.h_v + h];
      }
      float rk = 1.f, rq = p.scale;
      if (p.l2norm) {
        rk = 1.f / sqrtf(warp_sum(dot4(k, k, 0.f)) + 1e-6f);
        if (want_o) rq *= 1.f / sqrtf(warp_sum(dot4(q, q, 0.f)) + 1e-6f);
      }
      k = scale4(k, rk);
      q = scale4(q, rq);
      *reinterpret_cast<float4*>(&ks[warp][4 * lane]) = k;
      *reinterpret_cast<float4*>(&qs[warp][4 * lane]) = q;
    }
    __syncthreads();
    // Products of the window's keys with its keys and queries: eight lanes a pair.
#pragma unroll 1
    for (int e0 = 4 * warp; e0 < W * W; e0 += 4 * NW) {
      const int e = min(e0 + (lane >> 3), W * W - 1), a = e % W, t = e / W;
      uint64_t x2 = 0, y2 = 0;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(&ks[a][col0 + 32 * j]);
        const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&ks[t][col0 + 32 * j]);
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&qs[t][col0 + 32 * j]);
        x2 = fma2(u.y, k.y, fma2(u.x, k.x, x2));
        y2 = fma2(u.y, q.y, fma2(u.x, q.x, y2));
      }
      float x = pair_sum(x2), y = pair_sum(y2);
#pragma unroll
      for (int o = 1; o <= 4; o <<= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
      }
      if ((lane & 7) == 0 && a <= t && t < m) {
        float R = 1.f;
        for (int j = a + 1; j <= t; ++j) R *= alpha[j];
        kk[t][a] = R * x;
        kq[t][a] = R * y;
      }
    }
    // a_t = S k_t and b_t = S q_t: this lane's columns for all its rows, then the sums over a row's
    // eight lanes; with two rows, half of the lanes end up with each.
    float am[W], bm[W], d[W];
#pragma unroll
    for (int t = 0; t < W; ++t) {
      am[t] = bm[t] = 0.f;
      if (t >= m) continue;
      if (DELTA) am[t] = row_sum(&ks[t][col0]);
      if (want_o) bm[t] = row_sum(&qs[t][col0]);
    }
    __syncthreads();  // kk, kq
    float c = 1.f;
#pragma unroll
    for (int t = 0; t < W; ++t) {
      d[t] = 0.f;
      if (t >= m) continue;
      c *= alpha[t];
      float x = v[t];
      if (DELTA) {
        x = fmaf(-c, am[t], x);
#pragma unroll
        for (int e = 0; e < t; ++e) x = fmaf(-kk[t][e], d[e], x);
      }
      d[t] = beta[t] * x;
      if (want_o) {
        float o = c * bm[t];
#pragma unroll
        for (int e = 0; e <= t; ++e) o = fmaf(kq[t][e], d[e], o);
        // (of the lanes that hold the row's sums, another one writes each token)
        if ((lane & 3) == (t & 3) && (RG == 2 || (lane & 4) == 0) && my_row < p.d_v)
          store1(op + ((tok0 + t) * p.h_v + h) * p.d_v + my_row, o);
      }
    }
    if (p.keep && t0 + W >= cnt) return;
    // S <- c S + sum_t R_t d_t k_t^T
    float R = 1.f;
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
      for (int j = 0; j < J; ++j) s[r][j] = scale4(s[r][j], c);
#pragma unroll
    for (int t = W - 1; t >= 0; --t) {
      if (t >= m) continue;
      const float x = R * d[t], y = RG == 2 ? __shfl_xor_sync(0xffffffffu, x, 4) : 0.f;
      R *= alpha[t];
      const float x0 = my_r ? y : x, x1 = my_r ? x : y;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float4 k = *reinterpret_cast<const float4*>(&ks[t][col0 + 32 * j]);
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          const float f = r == 0 ? x0 : x1;
          s[r][j] = make_float4(fmaf(f, k.x, s[r][j].x), fmaf(f, k.y, s[r][j].y), fmaf(f, k.z, s[r][j].z),
                                fmaf(f, k.w, s[r][j].w));
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = row0 + 4 * r, col = col0 + 32 * j;
      if (row < p.d_v && col < p.d_k) __stcs(reinterpret_cast<float4*>(Sb + (size_t)row * p.d_k + col), s[r][j]);
    }
}

template <typename Tin, int J, int W, int RG, bool DELTA>
cudaError_t launch(const DecodeParams& p, cudaStream_t stream) {
  constexpr int NT = threads_of(W), rows = NT / 32 * 4 * RG;
  const dim3 grid(p.n, p.h_v, (p.d_v + rows - 1) / rows);
  decode_kernel<Tin, J, W, RG, DELTA><<<grid, NT, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename Tin, int J, int W>
cudaError_t launch_rows(const DecodeParams& p, cudaStream_t stream) {
  // Few states: 32 rows a CTA instead of 64, so that more SMs take part (one request of 32 heads, one
  // token: 3.5 us against 4.4; four: 5.1 against 5.3; eight, 256 states: 9.7 against 8.8).  152: the SMs.
  const bool few = (long long)p.n * p.h_v < 152;
  if (p.family == kDelta) return few ? launch<Tin, J, W, 1, true>(p, stream) : launch<Tin, J, W, 2, true>(p, stream);
  return few ? launch<Tin, J, W, 1, false>(p, stream) : launch<Tin, J, W, 2, false>(p, stream);
}

template <typename Tin>
cudaError_t launch_shape(const DecodeParams& p, cudaStream_t stream) {
  if (p.d_k <= 64)
    return p.window == 1 ? launch_rows<Tin, 2, 1>(p, stream)
           : p.window <= 4 ? launch_rows<Tin, 2, 4>(p, stream) : launch_rows<Tin, 2, 8>(p, stream);
  return p.window == 1 ? launch_rows<Tin, 4, 1>(p, stream)
         : p.window <= 4 ? launch_rows<Tin, 4, 4>(p, stream) : launch_rows<Tin, 4, 8>(p, stream);
}

}  // namespace

cudaError_t launch_decode(const DecodeParams& p, int bf16, cudaStream_t stream) {
  return bf16 ? launch_shape<__nv_bfloat16>(p, stream) : launch_shape<float>(p, stream);
}

}  // namespace gdn
