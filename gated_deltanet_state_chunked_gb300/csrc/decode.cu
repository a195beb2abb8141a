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
// Bound: HBM, 8 d_k d_v bytes per (request, v-head), for single tokens (256 requests, 32 heads of 128:
// 161 us, 97% of the rate of a copy).  Windows are bound by the latency of their steps (rows, products
// of the window, sums, the triangular solve) with two states at a time on an SM, and their instructions:
// 64 windows of 5 tokens, 32 heads of 128, take 41 us with outputs (20 us of reading) and 56 us
// committed (38 us of traffic), 43 and 57 us as whole calls.
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ float pair_sum(uint64_t x) {
  float a, b;
  unpair(x, a, b);
  return a + b;
}
__device__ __forceinline__ float4 scale4(float4 a, float s) { return make_float4(a.x * s, a.y * s, a.z * s, a.w * s); }
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Where a request's state is and how many of its tokens count; false: nothing to do.  Two requests on
// one slot would race on its state: the first that updates it has it, the others are skipped and
// reported (no_duplicate, while the state's loads are in flight).
__device__ __forceinline__ bool request(const DecodeParams& p, int i, int& slot, int& cnt) {
  slot = p.slots ? p.slots[i] : i;
  if (slot < 0) return false;  // padding
  cnt = p.counts ? p.counts[i] : p.window;
  if (slot >= p.n_slots || cnt < 0 || cnt > p.window) {
    if (threadIdx.x == 0) atomicExch(p.status, GDN_ERR_SHAPE);
    return false;
  }
  return cnt > 0;
}
template <int NT>
__device__ __forceinline__ bool no_duplicate(const DecodeParams& p, int i, int slot) {
  if (!p.slots || p.keep) return true;
  int dup = 0;
  for (int j = threadIdx.x; j < i; j += NT)
    dup |= p.slots[j] == slot && (!p.counts || (p.counts[j] > 0 && p.counts[j] <= p.window));
  if (!__syncthreads_or(dup)) return true;
  if (threadIdx.x == 0) atomicExch(p.status, GDN_ERR_SHAPE);
  return false;
}

// One token.  J: column groups of 32 (d_k at most 32 J); RG: groups of four rows per warp (1 or 2).
// 32 warps per SM at 64 registers a thread: what this kernel needs most is loads in flight (256 requests
// of 32 heads: 161 us; with another layout of the sums 171 us, against 176 us at 24 warps and 216 us at 16).
constexpr int kTokenNT = 256;
template <typename Tin, int J, int RG, bool DELTA>
__global__ void __launch_bounds__(kTokenNT, 4) decode_token_kernel(const DecodeParams p) {
  constexpr int NW = kTokenNT / 32;
  __shared__ __align__(16) float ks[kMaxHead], qs[kMaxHead];  // normalised, queries times scale
  __shared__ float s_alpha, s_beta, s_kq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x, h = blockIdx.y;
  int slot, cnt;
  if (!request(p, i, slot, cnt)) return;
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
  if (!no_duplicate<kTokenNT>(p, i, slot)) return;
  const bool want_o = !p.state_only;
  // the row whose sums this lane ends up with
  const bool second = RG == 2 && (lane & 4);
  const int my_row = row0 + (second ? 4 : 0);
  const float v = my_row < p.d_v ? load1(static_cast<const Tin*>(p.v) + ((size_t)i * p.h_v + h) * p.d_v + my_row) : 0.f;
  if (warp == 0) {
    const size_t at = ((size_t)i * p.h_k + h / p.v_per_k) * p.d_k + 4 * lane;
    float4 k = make_float4(0.f, 0.f, 0.f, 0.f), q = k;
    if (4 * lane < p.d_k) {
      k = load4(static_cast<const Tin*>(p.k) + at);
      if (want_o) q = load4(static_cast<const Tin*>(p.q) + at);
    }
    float rk = 1.f, rq = p.scale;
    if (p.l2norm) {
      rk = 1.f / sqrtf(warp_sum(dot4(k, k, 0.f)) + 1e-6f);
      if (want_o) rq *= 1.f / sqrtf(warp_sum(dot4(q, q, 0.f)) + 1e-6f);
    }
    k = scale4(k, rk);
    q = scale4(q, rq);
    *reinterpret_cast<float4*>(&ks[4 * lane]) = k;
    *reinterpret_cast<float4*>(&qs[4 * lane]) = q;
    const float kq = want_o ? warp_sum(dot4(k, q, 0.f)) : 0.f;
    if (lane == 0) {
      s_alpha = expf(p.family == kHeadDecay ? p.g[h] : p.g[(size_t)i * p.h_v + h]);
      s_beta = p.family == kHeadDecay ? 1.f : p.beta[(size_t)i * p.h_v + h];
      s_kq = kq;
    }
  }
  __syncthreads();
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
    float z = (second ? y[RG - 1] : y[0]) + __shfl_xor_sync(0xffffffffu, RG == 2 && !second ? y[RG - 1] : y[0], 4);
    z += __shfl_xor_sync(0xffffffffu, z, 2);
    return z + __shfl_xor_sync(0xffffffffu, z, 1);
  };
  const float alpha = s_alpha;
  const float d = s_beta * (DELTA ? fmaf(-alpha, row_sum(&ks[col0]), v) : v);
  if (want_o) {
    const float o = fmaf(s_kq, d, alpha * row_sum(&qs[col0]));
    if ((lane & 3) == 0 && (RG == 2 || (lane & 4) == 0) && my_row < p.d_v)
      store1(static_cast<Tin*>(p.O) + ((size_t)i * p.h_v + h) * p.d_v + my_row, o);
  }
  if (p.keep) return;
  const float other = RG == 2 ? __shfl_xor_sync(0xffffffffu, d, 4) : 0.f;
  const float d0 = second ? other : d, d1 = second ? d : other;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float4 k = *reinterpret_cast<const float4*>(&ks[col0 + 32 * j]);
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      const float f = r == 0 ? d0 : d1;
      const int row = row0 + 4 * r, col = col0 + 32 * j;
      const float4 u = scale4(s[r][j], alpha);
      if (row < p.d_v && col < p.d_k)
        __stcs(reinterpret_cast<float4*>(Sb + (size_t)row * p.d_k + col),
               make_float4(fmaf(f, k.x, u.x), fmaf(f, k.y, u.y), fmaf(f, k.z, u.z), fmaf(f, k.w, u.w)));
    }
  }
}

// A window, W tokens at once.  J as above; RG: groups of four rows per warp (1 or 4).  Four groups take
// 128 registers a thread and half the warps of two, but a token's row and the reductions serve twice the
// rows (64 windows of 5 tokens with outputs: 57 us against 70).  A token that does not count has zero
// keys and queries, alpha = 1 and beta = 0, so that nothing branches on it and the tokens' sums are under
// way together (45 us against 55).
__host__ __device__ constexpr int blocks_of(int RG, int NT) { return (RG == 4 ? 512 : 1024) / NT; }
template <typename Tin, int J, int W, int RG, int NT, bool DELTA>
__global__ void __launch_bounds__(NT, blocks_of(RG, NT)) decode_window_kernel(const DecodeParams p) {
  constexpr int NW = NT / 32, kPairs = W * (W + 1) / 2;
  static_assert(RG == 1 || RG == 4, "rows that share eight lanes");
  __shared__ __align__(16) float ks[W][kMaxHead], qs[W][kMaxHead];  // normalised, queries times scale
  __shared__ float alpha[W], beta[W];
  __shared__ float kk[kPairs], kq[kPairs];  // [t (t + 1) / 2 + i]: k_i.k_t and k_i.q_t times R_it
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x, h = blockIdx.y;
  int slot, cnt;
  if (!request(p, i, slot, cnt)) return;
  const int hk = h / p.v_per_k;
  const int col0 = 4 * (lane & 7);
  const int row0 = blockIdx.z * (NW * 4 * RG) + warp * (4 * RG) + (lane >> 3);
  float* Sb = p.S + ((size_t)slot * p.h_v + h) * p.d_v * p.d_k;
  const bool want_o = !p.state_only;
  const Tin* qp = static_cast<const Tin*>(p.q);
  const Tin* kp = static_cast<const Tin*>(p.k);
  const Tin* vp = static_cast<const Tin*>(p.v);
  Tin* op = static_cast<Tin*>(p.O);
  // the row whose sums this lane ends up with
  const bool hi4 = RG == 4 && (lane & 4), hi2 = RG == 4 && (lane & 2);
  const int my_row = row0 + (hi4 ? 8 : 0) + (hi2 ? 4 : 0);
  // The tokens' rows, ahead of the state's: they are needed first.
  constexpr int kPer = (W + NW - 1) / NW;  // tokens that a warp prepares
  float4 k_in[kPer], q_in[kPer];
  float g_in[kPer], b_in[kPer], v[W];
  auto fetch = [&](int t0) {
    const int m = min(W, cnt - t0);
    const size_t tok0 = (size_t)i * p.window + t0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int t = warp + NW * e;
      const size_t tok = tok0 + t;
      k_in[e] = q_in[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      g_in[e] = b_in[e] = 0.f;
      if (t < m) {
        if (4 * lane < p.d_k) {
          k_in[e] = load4(kp + (tok * p.h_k + hk) * p.d_k + 4 * lane);
          if (want_o) q_in[e] = load4(qp + (tok * p.h_k + hk) * p.d_k + 4 * lane);
        }
        if (lane == 0) {
          g_in[e] = p.family == kHeadDecay ? p.g[h] : p.g[tok * p.h_v + h];
          b_in[e] = p.family == kHeadDecay ? 1.f : p.beta[tok * p.h_v + h];
        }
      }
    }
    const Tin* at = vp + (tok0 * p.h_v + h) * p.d_v + my_row;
    const size_t step = (size_t)p.h_v * p.d_v;
#pragma unroll
    for (int t = 0; t < W; ++t) {
      v[t] = t < m && my_row < p.d_v ? load1(at) : 0.f;
      at += step;
    }
  };
  fetch(0);
  ulonglong2 s[RG][J];  // four columns, two by two
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = row0 + 4 * r, col = col0 + 32 * j;
      const float4 u = (row < p.d_v && col < p.d_k) ? __ldcs(reinterpret_cast<const float4*>(Sb + (size_t)row * p.d_k + col))
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
      s[r][j] = make_ulonglong2(pair(u.x, u.y), pair(u.z, u.w));
    }
  if (!no_duplicate<NT>(p, i, slot)) return;
  // products of this lane group's rows with x (this lane's columns), summed over a row's eight lanes;
  // with four rows, two of the lanes end up with each
  auto row_sum = [&](const float* x) {
    uint64_t y2[RG];
#pragma unroll
    for (int r = 0; r < RG; ++r) y2[r] = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(x + 32 * j);
#pragma unroll
      for (int r = 0; r < RG; ++r) y2[r] = fma2(s[r][j].y, u.y, fma2(s[r][j].x, u.x, y2[r]));
    }
    float z;
    if constexpr (RG == 4) {
      float y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = pair_sum(y2[r]);
      const float z0 = (hi4 ? y[2] : y[0]) + __shfl_xor_sync(0xffffffffu, hi4 ? y[0] : y[2], 4);
      const float z1 = (hi4 ? y[3] : y[1]) + __shfl_xor_sync(0xffffffffu, hi4 ? y[1] : y[3], 4);
      z = (hi2 ? z1 : z0) + __shfl_xor_sync(0xffffffffu, hi2 ? z0 : z1, 2);
    } else {
      z = pair_sum(y2[0]);
      z += __shfl_xor_sync(0xffffffffu, z, 4);
      z += __shfl_xor_sync(0xffffffffu, z, 2);
    }
    return z + __shfl_xor_sync(0xffffffffu, z, 1);
  };
  for (int t0 = 0; t0 < cnt; t0 += W) {
    const int m = min(W, cnt - t0);
    const size_t tok0 = (size_t)i * p.window + t0;
    if (t0 > 0) {
      fetch(t0);
      __syncthreads();  // the tables of the tokens before are read
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int t = warp + NW * e;
      if (t < W) {
        const float4 k = k_in[e], q = q_in[e];
        float rk = 1.f, rq = p.scale;
        if (p.l2norm) {
          rk = 1.f / sqrtf(warp_sum(dot4(k, k, 0.f)) + 1e-6f);
          if (want_o) rq *= 1.f / sqrtf(warp_sum(dot4(q, q, 0.f)) + 1e-6f);
        }
        *reinterpret_cast<float4*>(&ks[t][4 * lane]) = scale4(k, rk);
        *reinterpret_cast<float4*>(&qs[t][4 * lane]) = scale4(q, rq);
        if (lane == 0) {
          alpha[t] = expf(g_in[e]);
          beta[t] = b_in[e];
        }
      }
    }
    __syncthreads();
    // Products of the window's keys with its keys and queries, e = t (t + 1) / 2 + a: eight lanes a pair.
#pragma unroll 1
    for (int e0 = 4 * warp; e0 < kPairs; e0 += 4 * NW) {
      const int e = min(e0 + (lane >> 3), kPairs - 1);
      int t = 0;
#pragma unroll
      for (int u = 1; u < W; ++u) t += e >= u * (u + 1) / 2;
      const int a = e - t * (t + 1) / 2;
      uint64_t x2 = 0, y2 = 0;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(&ks[a][col0 + 32 * j]);
        const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&ks[t][col0 + 32 * j]);
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&qs[t][col0 + 32 * j]);
        x2 = fma2(u.y, k.y, fma2(u.x, k.x, x2));
        y2 = fma2(u.y, q.y, fma2(u.x, q.x, y2));
      }
      float x = pair_sum(x2), y = pair_sum(y2), R = 1.f;
#pragma unroll
      for (int o = 1; o <= 4; o <<= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
      }
#pragma unroll
      for (int j = 1; j < W; ++j) R *= j > a && j <= t ? alpha[j] : 1.f;
      if ((lane & 7) == 0) {
        kk[e] = R * x;
        kq[e] = R * y;
      }
    }
    // a_t = S k_t and b_t = S q_t
    float am[W], bm[W], d[W];
#pragma unroll
    for (int t = 0; t < W; ++t) am[t] = DELTA ? row_sum(&ks[t][col0]) : 0.f;
    if (want_o) {
#pragma unroll
      for (int t = 0; t < W; ++t) bm[t] = row_sum(&qs[t][col0]);
    }
    __syncthreads();  // kk, kq
    float c = 1.f;
#pragma unroll
    for (int t = 0; t < W; ++t) {
      c *= alpha[t];
      float x = v[t];
      if (DELTA) {
        x = fmaf(-c, am[t], x);
#pragma unroll
        for (int e = 0; e < t; ++e) x = fmaf(-kk[t * (t + 1) / 2 + e], d[e], x);
      }
      d[t] = t < m ? beta[t] * x : 0.f;
      if (want_o) bm[t] *= c;
    }
    if (want_o) {
      Tin* at = op + (tok0 * p.h_v + h) * p.d_v + my_row;
      const size_t step = (size_t)p.h_v * p.d_v;
#pragma unroll
      for (int t = 0; t < W; ++t) {
        float o = bm[t];
#pragma unroll
        for (int e = 0; e <= t; ++e) o = fmaf(kq[t * (t + 1) / 2 + e], d[e], o);
        // (of the lanes that hold the row's sums, another one writes each token)
        constexpr int kSame = RG == 4 ? 1 : 7;
        if (t < m && (lane & kSame) == (t & kSame) && my_row < p.d_v) store1(at, o);
        at += step;
      }
    }
    if (p.keep && t0 + W >= cnt) return;
    // S <- c S + sum_t R_t d_t k_t^T
    float R = 1.f;
    const uint64_t c2 = pair(c, c);
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
      for (int j = 0; j < J; ++j) s[r][j] = make_ulonglong2(mul2(s[r][j].x, c2), mul2(s[r][j].y, c2));
#pragma unroll
    for (int t = W - 1; t >= 0; --t) {
      float x[RG];  // R_tw d_t of every row
      x[0] = R * d[t];
      R *= alpha[t];
      if constexpr (RG == 4) {
        const float y0 = x[0], y1 = __shfl_xor_sync(0xffffffffu, y0, 2);
        const float z0 = hi2 ? y1 : y0, z1 = hi2 ? y0 : y1;  // rows 0 and 1, or 2 and 3
        const float u0 = __shfl_xor_sync(0xffffffffu, z0, 4), u1 = __shfl_xor_sync(0xffffffffu, z1, 4);
        x[0] = hi4 ? u0 : z0;
        x[1] = hi4 ? u1 : z1;
        x[2] = hi4 ? z0 : u0;
        x[3] = hi4 ? z1 : u1;
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&ks[t][col0 + 32 * j]);
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          const uint64_t f = pair(x[r], x[r]);
          s[r][j] = make_ulonglong2(fma2(f, k.x, s[r][j].x), fma2(f, k.y, s[r][j].y));
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = row0 + 4 * r, col = col0 + 32 * j;
      float4 u;
      unpair(s[r][j].x, u.x, u.y);
      unpair(s[r][j].y, u.z, u.w);
      if (row < p.d_v && col < p.d_k) __stcs(reinterpret_cast<float4*>(Sb + (size_t)row * p.d_k + col), u);
    }
}

dim3 grid_of(const DecodeParams& p, int rows) { return dim3(p.n, p.h_v, (p.d_v + rows - 1) / rows); }

template <typename Tin, int J, bool DELTA>
void launch_token(const DecodeParams& p, bool few, cudaStream_t stream) {
  if (few) decode_token_kernel<Tin, J, 1, DELTA><<<grid_of(p, kTokenNT / 8), kTokenNT, 0, stream>>>(p);
  else decode_token_kernel<Tin, J, 2, DELTA><<<grid_of(p, kTokenNT / 4), kTokenNT, 0, stream>>>(p);
}

// CTAs of 64 rows (four warps) for heads of up to 64 rows, where half of eight warps would idle (64
// windows of 5 tokens, 64 x 64 heads: 19 us against 37), and for windows of up to 4 tokens, where four
// CTAs an SM overlap better (of 2: 46 us against 50; of 4: 52 against 56); 128 rows for longer ones,
// whose products would be computed twice (of 5: 42 us against 52).
template <typename Tin, int J, int W, bool DELTA>
void launch_window(const DecodeParams& p, bool few, cudaStream_t stream) {
  if (few) {
    decode_window_kernel<Tin, J, W, 1, 512, DELTA><<<grid_of(p, 64), 512, 0, stream>>>(p);
    return;
  }
  if constexpr (W > 4) {
    if (p.d_v > 64) {
      decode_window_kernel<Tin, J, W, 4, 256, DELTA><<<grid_of(p, 128), 256, 0, stream>>>(p);
      return;
    }
  }
  decode_window_kernel<Tin, J, W, 4, 128, DELTA><<<grid_of(p, 64), 128, 0, stream>>>(p);
}

template <typename Tin, int J, bool DELTA>
void launch_length(const DecodeParams& p, cudaStream_t stream) {
  // Few states: fewer rows a CTA, so that more SMs take part (one request of 32 heads, one token: 3.5 us
  // against 4.4; four: 5.1 against 5.3; eight, 256 states: 9.7 against 8.8).  152: the SMs.  Windows are
  // unrolled at their own length up to 6 tokens, longer ones eight tokens at a time.
  const bool few = (long long)p.n * p.h_v < 152;
  switch (p.window) {
    case 1: return launch_token<Tin, J, DELTA>(p, few, stream);
    case 2: return launch_window<Tin, J, 2, DELTA>(p, few, stream);
    case 3: return launch_window<Tin, J, 3, DELTA>(p, few, stream);
    case 4: return launch_window<Tin, J, 4, DELTA>(p, few, stream);
    case 5: return launch_window<Tin, J, 5, DELTA>(p, few, stream);
    case 6: return launch_window<Tin, J, 6, DELTA>(p, few, stream);
    default: return launch_window<Tin, J, 8, DELTA>(p, few, stream);
  }
}

template <typename Tin>
cudaError_t launch_shape(const DecodeParams& p, cudaStream_t stream) {
  if (p.family == kDelta) p.d_k <= 64 ? launch_length<Tin, 2, true>(p, stream) : launch_length<Tin, 4, true>(p, stream);
  else p.d_k <= 64 ? launch_length<Tin, 2, false>(p, stream) : launch_length<Tin, 4, false>(p, stream);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode(const DecodeParams& p, int bf16, cudaStream_t stream) {
  return bf16 ? launch_shape<__nv_bfloat16>(p, stream) : launch_shape<float>(p, stream);
}

}  // namespace gdn
