// Linear attention with a decay for each head over packed prompts, on the CUDA cores in fp32: fp32
// inputs of any head size.
//
// Method: the scalar-decay family that "LinearKV: One Cached State Suffices for Position-Independent
// Caching in Hybrid LLMs" (composition passage) sets beside the delta rule, with a decay lambda_h that
// belongs to the head:  S_t = lambda_h S_{t-1} + v_t k_t^T,  o_t = S_t (scale q_t).  Chunk by chunk
// (64 tokens, n of them in the last one) with the entering state S:
//   P_ts = scale lambda^(t-s) q_t.k_s   (s <= t)
//   O_t  = sum_s P_ts v_s + scale lambda^(t+1) S q_t
//   S   <- lambda^n S + sum_s lambda^(n-1-s) v_s k_s^T
// One CTA owns 32 rows of one (sequence, v-head) state and walks the sequence's chunks.
#include <cuda_bf16.h>

#include "gdn_internal.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace {

using tcp::chunk_info;
using tcp::ChunkInfo;

constexpr int C = kChunk, R = 32, NT = 256;
constexpr int QS = kMaxHead + 4;  // row strides (floats) of the tiles
constexpr int PS = C + 4, VS = R + 4;

struct Smem {
  float Q[C * QS], K[C * QS], S[R * QS], P[C * PS], V[C * VS], W[C * VS];
  float pw[C + 1];  // lambda^n
  int scratch[32];
};

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

template <typename Tin>
__global__ void __launch_bounds__(NT) linear_simt_kernel(const LinearParams p) {
  extern __shared__ __align__(16) unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int seq = blockIdx.x, h = blockIdx.y, r0 = blockIdx.z * R;
  const int d_k = p.d_k, d_v = p.d_v, hk = h / (p.h_v / p.h_k);
  const ChunkInfo ci = chunk_info(p.cu, p.n_seqs, p.total_tokens, seq, -1, sm.scratch);
  if (!ci.valid) {
    if (tid == 0) atomicExch(p.status, GDN_ERR_SHAPE);
    return;
  }
  const int t_begin = p.cu[seq], t_end = p.cu[seq + 1];
  const float g = p.log_decay[h];
  for (int n = tid; n <= C; n += NT) sm.pw[n] = n ? expf((float)n * g) : 1.f;
  float* S_out = p.S_out + ((size_t)seq * p.h_v + h) * d_v * d_k;
  const float* S0 = p.S0 ? p.S0 + ((size_t)seq * p.h_v + h) * d_v * d_k : nullptr;
  for (int e = tid; e < R * d_k; e += NT) {
    const int r = e / d_k, c = e % d_k;
    sm.S[r * QS + c] = S0 && r0 + r < d_v ? S0[(size_t)(r0 + r) * d_k + c] : 0.f;
  }
  const Tin* q = static_cast<const Tin*>(p.q);
  const Tin* k = static_cast<const Tin*>(p.k);
  const Tin* v = static_cast<const Tin*>(p.v);
  Tin* O = static_cast<Tin*>(p.O);
  for (int t0 = t_begin; t0 < t_end; t0 += C) {
    const int n = min(C, t_end - t0);
    __syncthreads();
    for (int e = tid; e < C * d_k; e += NT) {
      const int t = e / d_k, c = e % d_k;
      const size_t at = ((size_t)(t0 + t) * p.h_k + hk) * d_k + c;
      sm.K[t * QS + c] = t < n ? load1(k + at) : 0.f;
      if (p.write_O) sm.Q[t * QS + c] = t < n ? load1(q + at) : 0.f;
    }
    for (int e = tid; e < C * R; e += NT) {
      const int t = e / R, r = e % R;
      const float x = t < n && r0 + r < d_v ? load1(v + ((size_t)(t0 + t) * p.h_v + h) * d_v + r0 + r) : 0.f;
      sm.V[t * VS + r] = x;
      sm.W[t * VS + r] = t < n ? x * sm.pw[n - 1 - t] : 0.f;
    }
    __syncthreads();
    if (p.write_O) {
      {  // P: rows ty + 16 a, columns tx + 16 b
        float acc[4][4] = {};
        for (int c = 0; c < d_k; c += 4) {
          float4 x[4], y[4];
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            x[a] = *reinterpret_cast<const float4*>(&sm.Q[(ty + 16 * a) * QS + c]);
            y[a] = *reinterpret_cast<const float4*>(&sm.K[(tx + 16 * a) * QS + c]);
          }
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 4; ++b) acc[a][b] = dot4(x[a], y[b], acc[a][b]);
        }
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int t = ty + 16 * a, s = tx + 16 * b;
            sm.P[t * PS + s] = s <= t ? acc[a][b] * sm.pw[t - s] : 0.f;
          }
      }
      __syncthreads();
      {  // O: rows ty + 16 a, value columns tx + 16 b
        float inter[4][2] = {}, intra[4][2] = {};
        for (int c = 0; c < d_k; c += 4) {
          float4 x[4], y[2];
#pragma unroll
          for (int a = 0; a < 4; ++a) x[a] = *reinterpret_cast<const float4*>(&sm.Q[(ty + 16 * a) * QS + c]);
#pragma unroll
          for (int b = 0; b < 2; ++b) y[b] = *reinterpret_cast<const float4*>(&sm.S[(tx + 16 * b) * QS + c]);
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) inter[a][b] = dot4(x[a], y[b], inter[a][b]);
        }
        for (int s = 0; s < C; ++s) {
          const float y0 = sm.V[s * VS + tx], y1 = sm.V[s * VS + tx + 16];
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const float x = sm.P[(ty + 16 * a) * PS + s];
            intra[a][0] = fmaf(x, y0, intra[a][0]);
            intra[a][1] = fmaf(x, y1, intra[a][1]);
          }
        }
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int t = ty + 16 * a, r = r0 + tx + 16 * b;
            if (t < n && r < d_v)
              store1(O + ((size_t)(t0 + t) * p.h_v + h) * d_v + r,
                     p.scale * fmaf(sm.pw[t + 1], inter[a][b], intra[a][b]));
          }
      }
      __syncthreads();  // every reader of S is done
    }
    {  // S: rows (tid >> 5) + 8 a, columns 4 (tid & 31) + [0, 4)
      const int c = 4 * (tid & 31), rr = tid >> 5;
      if (c < d_k) {
        float4 acc[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) acc[a] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < n; ++s) {
          const float4 y = *reinterpret_cast<const float4*>(&sm.K[s * QS + c]);
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const float x = sm.W[s * VS + rr + 8 * a];
            acc[a].x = fmaf(x, y.x, acc[a].x);
            acc[a].y = fmaf(x, y.y, acc[a].y);
            acc[a].z = fmaf(x, y.z, acc[a].z);
            acc[a].w = fmaf(x, y.w, acc[a].w);
          }
        }
        const DecayStep f = decay_step(g, n);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          float4* s = reinterpret_cast<float4*>(&sm.S[(rr + 8 * a) * QS + c]);
          *s = make_float4(f(s->x, acc[a].x), f(s->y, acc[a].y), f(s->z, acc[a].z), f(s->w, acc[a].w));
        }
      }
    }
  }
  __syncthreads();
  for (int e = tid; e < R * d_k; e += NT) {
    const int r = e / d_k, c = e % d_k;
    if (r0 + r < d_v) S_out[(size_t)(r0 + r) * d_k + c] = sm.S[r * QS + c];
  }
}

}  // namespace

cudaError_t launch_linear_simt(const LinearParams& p, int bf16, cudaStream_t stream) {
  auto kern = bf16 ? linear_simt_kernel<__nv_bfloat16> : linear_simt_kernel<float>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
  if (e != cudaSuccess) return e;
  const dim3 grid(p.n_seqs, p.h_v, (p.d_v + R - 1) / R);
  kern<<<grid, NT, sizeof(Smem), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
