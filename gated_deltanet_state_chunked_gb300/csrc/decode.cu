// Recurrent form on a pool of states: one token, or a short window of tokens, per request.
//
// Method: "Tail-Replay: Escaping the Curse of Linear Attention in Prefix Caching for Hybrid LLMs",
// section 2 Eq. (1), token by token; per v-head, with the state S (d_v x d_k) of the request:
//   delta rule     S <- alpha S (I - beta k k^T) + beta v k^T
//   scalar decay   S <- alpha S + beta v k^T
//   head decay     S <- lambda_h S + v k^T
// and the readout o = S (scale q) with the updated state.
//
// Every row s of S moves on its own: with a = s.k and b = s.q taken on the state before the token,
//   d = beta (v_r - alpha a)   (no alpha a outside the delta rule),   s <- alpha s + d k,
//   o_r = scale (alpha b + d k.q),
// so one token needs one round of reductions (a and b together) instead of two.
//
// Layout: eight lanes share a row, lane l holding columns 4 (l & 7) + 32 j + [0, 4), so a warp's load
// covers four rows in whole 128-byte lines and a reduction takes three shuffles.  A state is read once
// into registers and written once, whatever the window's length.  Bound: HBM, 8 d_k d_v bytes per
// (request, v-head) against about 6 d_k d_v flop a token.
#include <cuda_bf16.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int NW = 8;         // warps per CTA
constexpr int NT = 32 * NW;

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
// Sum over the eight lanes of a row.
__device__ __forceinline__ float sum8(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  return x;
}

// J: column groups of 32 (ceil(d_k / 32)); RG: groups of four rows per warp.
template <typename Tin, int J, int RG>
__global__ void __launch_bounds__(NT) decode_kernel(const DecodeParams p) {
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
      s[r][j] = (row < p.d_v && col < p.d_k) ? *reinterpret_cast<const float4*>(Sb + (size_t)row * p.d_k + col)
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  // Two requests on one slot would race on its state: the first of them has it, the others are
  // skipped and reported.  (Checked while the state's loads are in flight.)
  if (p.slots && !p.keep) {
    int dup = 0;
    for (int j = tid; j < i; j += NT) dup |= p.slots[j] == slot;
    if (__syncthreads_or(dup)) {
      if (tid == 0) atomicExch(p.status, GDN_ERR_SHAPE);
      return;
    }
  }
  const float head_alpha = p.family == kHeadDecay ? expf(p.g[h]) : 0.f;
  const Tin* qp = static_cast<const Tin*>(p.q);
  const Tin* kp = static_cast<const Tin*>(p.k);
  const Tin* vp = static_cast<const Tin*>(p.v);
  Tin* op = static_cast<Tin*>(p.O);
  for (int t = 0; t < cnt; ++t) {
    const size_t tok = (size_t)i * p.window + t;
    float4 k[J], q[J];
    float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int col = col0 + 32 * j;
      const bool in = col < p.d_k;
      k[j] = in ? load4(kp + (tok * p.h_k + hk) * p.d_k + col) : make_float4(0.f, 0.f, 0.f, 0.f);
      q[j] = in && !p.state_only ? load4(qp + (tok * p.h_k + hk) * p.d_k + col) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float v[RG];
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      const int row = row0 + 4 * r;
      v[r] = row < p.d_v ? load1(vp + (tok * p.h_v + h) * p.d_v + row) : 0.f;
    }
    const float alpha = p.family == kHeadDecay ? head_alpha : expf(p.g[tok * p.h_v + h]);
    const float beta = p.family == kHeadDecay ? 1.f : p.beta[tok * p.h_v + h];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      kk = dot4(k[j], k[j], kk);
      qq = dot4(q[j], q[j], qq);
      kq = dot4(k[j], q[j], kq);
    }
    kk = sum8(kk);
    qq = sum8(qq);
    kq = sum8(kq);
    const float rk = p.l2norm ? 1.f / sqrtf(kk + 1e-6f) : 1.f;
    const float rq = (p.l2norm ? 1.f / sqrtf(qq + 1e-6f) : 1.f) * p.scale;
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        a = dot4(s[r][j], k[j], a);
        b = dot4(s[r][j], q[j], b);
      }
      a = sum8(a) * rk;
      b = sum8(b);
      const float d = beta * (p.family == kDelta ? fmaf(-alpha, a, v[r]) : v[r]) * rk;  // along the raw key
#pragma unroll
      for (int j = 0; j < J; ++j) {
        s[r][j].x = fmaf(alpha, s[r][j].x, d * k[j].x);
        s[r][j].y = fmaf(alpha, s[r][j].y, d * k[j].y);
        s[r][j].z = fmaf(alpha, s[r][j].z, d * k[j].z);
        s[r][j].w = fmaf(alpha, s[r][j].w, d * k[j].w);
      }
      const int row = row0 + 4 * r;
      if (!p.state_only && (lane & 7) == 0 && row < p.d_v)
        store1(op + (tok * p.h_v + h) * p.d_v + row, rq * fmaf(alpha, b, d * kq));
    }
  }
  if (p.keep) return;
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = row0 + 4 * r, col = col0 + 32 * j;
      if (row < p.d_v && col < p.d_k) *reinterpret_cast<float4*>(Sb + (size_t)row * p.d_k + col) = s[r][j];
    }
}

template <typename Tin, int J, int RG>
cudaError_t launch(const DecodeParams& p, cudaStream_t stream) {
  const int rows = NW * 4 * RG;
  const dim3 grid(p.n, p.h_v, (p.d_v + rows - 1) / rows);
  decode_kernel<Tin, J, RG><<<grid, NT, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename Tin, int RG>
cudaError_t launch_cols(const DecodeParams& p, cudaStream_t stream) {
  switch ((p.d_k + 31) / 32) {
    case 1: return launch<Tin, 1, RG>(p, stream);
    case 2: return launch<Tin, 2, RG>(p, stream);
    case 3: return launch<Tin, 3, RG>(p, stream);
    default: return launch<Tin, 4, RG>(p, stream);
  }
}

}  // namespace

cudaError_t launch_decode(const DecodeParams& p, int bf16, cudaStream_t stream) {
  return bf16 ? launch_cols<__nv_bfloat16, 4>(p, stream) : launch_cols<float, 4>(p, stream);
}

}  // namespace gdn
