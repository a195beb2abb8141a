// Linear attention with a decay for each head over packed prompts, fp32 inputs, on the CUDA cores.
//
// Method: the scalar-decay family that "LinearKV: One Cached State Suffices for Position-Independent
// Caching in Hybrid LLMs" (composition passage) sets beside the delta rule, with a decay lambda_h that
// belongs to the head:  S_t = lambda_h S_{t-1} + v_t k_t^T,  o_t = S_t (scale q_t).  Chunk by chunk
// (64 tokens, n of them in the last one) with the entering state S:
//   P_ts = lambda^(t-s) q_t.k_s   (s <= t)
//   O_t  = scale (sum_s P_ts v_s + lambda^(t+1) S q_t)
//   S   <- lambda^n S + sum_s lambda^(n-1-s) v_s k_s^T
// One CTA owns a (segment, v-head) and walks its chunks.  The state stays in registers, up to 8 x 8
// entries a thread, and is copied to shared memory, transposed, as the readout's operand.  Every product
// is a register tile fed from shared memory: 4 x 4 for P (blocks above the diagonal skipped), 8 rows x 4
// columns for O, 8 x 8 for S.  Keys, values and the next chunk's keys rotate through three buffers: the
// values are weighted in place, and only their load waits for the end of a chunk.
//
// Bound: fp32 arithmetic and the shared-memory reads that feed it.  A chunk of 128 x 128 heads is 2.7 M
// multiply-adds, 21,300 clocks of an SM's pipes; it takes about 39,000 (P 7,000, Q S 12,700, P V 6,500,
// S 11,200), with the 8 warps that one CTA's shared memory leaves room for.  24 ragged prompts of 16,411
// tokens in all (8/16 heads, d_k 96, d_v 120): 465 to 495 us on different boards (on the first: the tiles read without asynchronous copies: 523;
// four multiply-adds where two packed ones are now: 478; rows of P V paired so that every warp has as many
// tokens, and packed scores: 469 to 471, though 4% less at 128 x 128; one row a thread and no tiles: 3,830).  TF32
// products on the warp-level tensor cores were not taken: three of them for fp32 accuracy run at 1.36 times
// this rate.
#include "linear_work.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace {

constexpr int C = kChunk, D = kMaxHead, NT = 256;
constexpr int TS = D + 4;  // row stride (floats) of Q, K, V and of the state's copy
constexpr int PS = C + 4;

struct Smem {
  float Q[C * TS], KV[3][C * TS], St[D * TS], P[C * PS];  // KV: keys, values, and the next chunk's keys, by turns
  float pw[C + 1];  // lambda^n
};

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
// Two fused multiply-adds in one instruction (values as register pairs): the same rate as two, but half
// the issue slots, which the loads beside them need.
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
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
// 16 bytes of global memory into shared memory, or zeros.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {
  const int bytes = there ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All copies are there but those of the last `left` groups.
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// JN: groups of 16 state columns (d_k at most 16 JN); RI: state rows a thread (d_v at most 16 RI), 8 or 4,
// and as many rows of O (at 4 a warp's halves take four rows each).
template <bool OUT, int JN, int RI>
__global__ void __launch_bounds__(NT, 1) linear_simt_kernel(const LinearWork p) {
  extern __shared__ __align__(16) unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, x = tid & 15, y = tid >> 4;
  const int h = blockIdx.x % p.h_v, u = blockIdx.x / p.h_v;
  tc::grid_dep_launch();
  // The plan; and no launch is over before the one ahead of it.  (Of a single sequence the segments with
  // outputs load their inputs first and wait below.)
  const bool later = OUT && !p.list;
  if (!later) tc::grid_dep_wait();
  const Segment seg = p.list ? p.list[u] : only_segment(p, u);
  if (!p.list && blockIdx.x == 0 && tid == 0 && seg.seq < 0) atomicExch(p.status, GDN_ERR_SHAPE);
  if (seg.seq < 0 || (p.local_only && seg.seg + 1 == seg.n_seg)) {
    tc::grid_dep_wait();
    return;
  }
  const ItemState state = item_state(p, seg, h, OUT);
  const int d_k = p.d_k, d_v = p.d_v, hk = h / (p.h_v / p.h_k);
  const float g = p.log_decay[h];
  const float* q = static_cast<const float*>(p.q) + (size_t)hk * d_k;
  const float* k = static_cast<const float*>(p.k) + (size_t)hk * d_k;
  const float* v = static_cast<const float*>(p.v) + (size_t)h * d_v;
  float* O = static_cast<float*>(p.O) + (size_t)h * d_v;
  const size_t qk_row = (size_t)p.h_k * d_k, v_row = (size_t)p.h_v * d_v;
  const int t_end = seg.t_begin + seg.len;

  // Rows [t0, t0 + 64) of a tensor into a tile; zero behind the segment's end and the head's width.
  auto load = [&](float* tile, const float* src, size_t row, int d, int t0) {
    for (int e = tid; e < C * (D / 4); e += NT) {
      const int t = e / (D / 4), c = 4 * (e % (D / 4));
      const bool there = t0 + t < t_end && c < d;
      copy16(tile + t * TS + c, there ? src + (size_t)(t0 + t) * row + c : src, there);
    }
  };
  if (seg.len > 0) {
    if (OUT) load(sm.Q, q, qk_row, d_k, seg.t_begin);
    load(sm.KV[0], k, qk_row, d_k, seg.t_begin);
    copies_commit();
    load(sm.KV[1], v, v_row, d_v, seg.t_begin);
  }
  copies_commit();
  for (int n = tid; n <= C; n += NT) sm.pw[n] = n ? expf((float)n * g) : 1.f;
  if (later) tc::grid_dep_wait();  // the entering states
  float s[RI][JN];  // rows RI y + i, columns x + 16 j
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < JN; ++j) {
      const int r = RI * y + i, c = x + 16 * j;
      s[i][j] = state.S_in && r < d_v && c < d_k ? state.S_in[(size_t)r * d_k + c] : 0.f;
    }
  auto publish_state = [&]() {
#pragma unroll
    for (int j = 0; j < JN; ++j) {
      float* at = sm.St + (x + 16 * j) * TS + RI * y;
#pragma unroll
      for (int i = 0; i < RI; i += 4)
        *reinterpret_cast<float4*>(at + i) = make_float4(s[i][j], s[i + 1][j], s[i + 2][j], s[i + 3][j]);
    }
  };
  if (OUT) publish_state();

  float *tk = sm.KV[0], *tv = sm.KV[1], *spare = sm.KV[2];
  for (int t0 = seg.t_begin; t0 < t_end; t0 += C) {
    const int n = min(C, t_end - t0);
    const bool more = t0 + C < t_end;
    copies_wait<1>();  // queries and keys (the values may still be on their way)
    __syncthreads();
    if (more) load(spare, k, qk_row, d_k, t0 + C);
    copies_commit();
    if (OUT) {
      {  // P: rows y + 16 a, columns x + 16 b; a block with b > a lies above the diagonal
        float acc[4][4] = {};
#pragma unroll 2
        for (int c = 0; c < d_k; c += 4) {
          float4 a4[4], b4[4];
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            a4[a] = *reinterpret_cast<const float4*>(&sm.Q[(y + 16 * a) * TS + c]);
            b4[a] = *reinterpret_cast<const float4*>(&tk[(x + 16 * a) * TS + c]);
          }
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b <= a; ++b) acc[a][b] = dot4(a4[a], b4[b], acc[a][b]);
        }
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int t = y + 16 * a, e = x + 16 * b;
            sm.P[t * PS + e] = e <= t ? acc[a][b] * sm.pw[t - e] : 0.f;
          }
      }
      copies_wait<1>();  // values (all but the next keys)
      __syncthreads();
      {  // O: rows row0 + i, columns col0 + [0, 4)
        const int row0 = 8 * warp + (RI == 4 ? 4 * (lane >> 4) : 0), col0 = 4 * (RI == 4 ? lane & 15 : lane);
        uint64_t o[RI][2];  // pairs of columns
#pragma unroll
        for (int i = 0; i < RI; ++i) o[i][0] = o[i][1] = 0;
        auto rank1 = [&](float a, ulonglong2 b, uint64_t (&c)[2]) {
          const uint64_t a2 = pair(a, a);
          c[0] = fma2(a2, b.x, c[0]);
          c[1] = fma2(a2, b.y, c[1]);
        };
#pragma unroll 2
        for (int c = 0; c < d_k; c += 4) {
          ulonglong2 b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) b[e] = *reinterpret_cast<const ulonglong2*>(&sm.St[(c + e) * TS + col0]);
#pragma unroll
          for (int i = 0; i < RI; ++i) {
            const float4 a = *reinterpret_cast<const float4*>(&sm.Q[(row0 + i) * TS + c]);
            rank1(a.x, b[0], o[i]);
            rank1(a.y, b[1], o[i]);
            rank1(a.z, b[2], o[i]);
            rank1(a.w, b[3], o[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < RI; ++i) {
          const float f = sm.pw[row0 + i + 1];
#pragma unroll
          for (int e = 0; e < 2; ++e) o[i][e] = fma2(pair(f, f), o[i][e], 0);
        }
#pragma unroll 2
        for (int e0 = 0; e0 < 8 * warp; e0 += 4) {
          ulonglong2 b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) b[e] = *reinterpret_cast<const ulonglong2*>(&tv[(e0 + e) * TS + col0]);
#pragma unroll
          for (int i = 0; i < RI; ++i) {
            const float4 a = *reinterpret_cast<const float4*>(&sm.P[(row0 + i) * PS + e0]);
            rank1(a.x, b[0], o[i]);
            rank1(a.y, b[1], o[i]);
            rank1(a.z, b[2], o[i]);
            rank1(a.w, b[3], o[i]);
          }
        }
        // The warp's own eight tokens: a later one is left out, not multiplied by a score of zero (its
        // value may be infinite).
#pragma unroll
        for (int e0 = 0; e0 < 8; e0 += 4) {
          ulonglong2 b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) b[e] = *reinterpret_cast<const ulonglong2*>(&tv[(8 * warp + e0 + e) * TS + col0]);
#pragma unroll
          for (int i = 0; i < RI; ++i) {
            const int last = row0 + i - 8 * warp - e0;  // of these four tokens, the last that is not later
            const float4 a = *reinterpret_cast<const float4*>(&sm.P[(row0 + i) * PS + 8 * warp + e0]);
            if (0 <= last) rank1(a.x, b[0], o[i]);
            if (1 <= last) rank1(a.y, b[1], o[i]);
            if (2 <= last) rank1(a.z, b[2], o[i]);
            if (3 <= last) rank1(a.w, b[3], o[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < RI; ++i) {
          const int t = row0 + i;
          float a, b, c, d;
          unpair(o[i][0], a, b);
          unpair(o[i][1], c, d);
          if (t < n && col0 < d_v)
            *reinterpret_cast<float4*>(O + (size_t)(t0 + t) * v_row + col0) =
                make_float4(p.scale * a, p.scale * b, p.scale * c, p.scale * d);
        }
      }
      __syncthreads();  // Q and the state's copy are read
      if (more) load(sm.Q, q, qk_row, d_k, t0 + C);
    } else {
      copies_wait<1>();
      __syncthreads();
    }
    copies_commit();
    // the values times their weights, in place
    for (int e = tid; e < n * (D / 4); e += NT) {
      float4* at = reinterpret_cast<float4*>(&tv[e / (D / 4) * TS + 4 * (e % (D / 4))]);
      const float w = sm.pw[n - 1 - e / (D / 4)];
      *at = make_float4(w * at->x, w * at->y, w * at->z, w * at->w);
    }
    __syncthreads();
    {  // S
      uint64_t acc[RI / 2][JN] = {};  // pairs of rows
#pragma unroll 4
      for (int e = 0; e < n; ++e) {
        uint64_t a[RI / 2];
#pragma unroll
        for (int i = 0; i < RI; i += 4) {
          const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&tv[e * TS + RI * y + i]);
          a[i / 2] = f.x;
          a[i / 2 + 1] = f.y;
        }
#pragma unroll
        for (int j = 0; j < JN; ++j) {
          const float b = tk[e * TS + x + 16 * j];
          const uint64_t b2 = pair(b, b);
#pragma unroll
          for (int i = 0; i < RI / 2; ++i) acc[i][j] = fma2(a[i], b2, acc[i][j]);
        }
      }
      const DecayStep f = decay_step(g, n);
#pragma unroll
      for (int i = 0; i < RI / 2; ++i)
#pragma unroll
        for (int j = 0; j < JN; ++j) {
          float d0, d1;
          unpair(acc[i][j], d0, d1);
          s[2 * i][j] = f(s[2 * i][j], d0);
          s[2 * i + 1][j] = f(s[2 * i + 1][j], d1);
        }
    }
    if (more) {
      if (OUT) publish_state();
      __syncthreads();  // the keys and values are read
      load(tk, v, v_row, d_v, t0 + C);
      copies_commit();
      float* const old = tv;  // (free: the keys' next but one place)
      tv = tk;
      tk = spare;
      spare = old;
    }
  }
  if (state.dst < 0) return;
  float* dst = (state.to_local ? p.local : p.S_out) + (size_t)state.dst * d_v * d_k;
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < JN; ++j) {
      const int r = RI * y + i, c = x + 16 * j;
      if (r < d_v && c < d_k) dst[(size_t)r * d_k + c] = s[i][j];
    }
}

template <bool OUT, int JN, int RI>
cudaError_t launch_items(const LinearWork& p, int units, cudaStream_t stream) {
  const cudaError_t e =
      cudaFuncSetAttribute(linear_simt_kernel<OUT, JN, RI>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units * p.h_v);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = sizeof(Smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, linear_simt_kernel<OUT, JN, RI>, p);
}

template <bool OUT, int RI>
cudaError_t launch_columns(const LinearWork& p, int units, cudaStream_t stream) {
  if (p.d_k <= 64) return launch_items<OUT, 4, RI>(p, units, stream);
  if (p.d_k <= 96) return launch_items<OUT, 6, RI>(p, units, stream);
  return launch_items<OUT, 8, RI>(p, units, stream);
}

template <bool OUT>
cudaError_t launch_shape(const LinearWork& p, int units, cudaStream_t stream) {
  return p.d_v <= 64 ? launch_columns<OUT, 4>(p, units, stream) : launch_columns<OUT, 8>(p, units, stream);
}

}  // namespace

cudaError_t launch_linear_simt_items(const LinearWork& p, bool out, int units, cudaStream_t stream) {
  return out ? launch_shape<true>(p, units, stream) : launch_shape<false>(p, units, stream);
}

}  // namespace gdn
