// gdn_paged_attn on the CUDA cores.
#include "paged_work.cuh"

namespace gdn {
namespace paged {
namespace {

// One CTA of 256 threads, tiles of BM = 16 TR query rows x 64 keys.  Thread (ty, tx) = (tid / 16, tid % 16)
// holds rows TR ty .. and keys tx + 16 j of the scores, columns 4 tx + 64 j of the outputs.  Keys and values each
// have one buffer: the next tile's keys arrive while the values are multiplied, its values while the scores are.
constexpr int NT = 256, BN = 64, LDP = BN + 4;

__device__ __forceinline__ void cp16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four values of a row of the pages (or zeros) into shared memory.
__device__ __forceinline__ void put4(float* dst, const float* src, bool there) { cp16(dst, src, there); }
__device__ __forceinline__ void put4(float* dst, const __nv_bfloat16* src, bool there) {
  float4 v = {0.f, 0.f, 0.f, 0.f};
  if (there) {
    const uint2 u = *reinterpret_cast<const uint2*>(src);
    v = float4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
               __uint_as_float(u.y & 0xffff0000u)};
  }
  *reinterpret_cast<float4*>(dst) = v;
}

template <typename T>
__device__ __forceinline__ void load_tile(const PagedParams& p, float* dst, int ld, const T* base, int64_t page_step,
                                          int64_t token_step, int req, int j0, const Span& span) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mask = (1 << p.page_shift) - 1;
  int page[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = j0 + warp * 8 + i;
    page[i] = j >= span.lo && j < span.hi ? page_of(p, req, j) : -1;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = warp * 8 + i;
    const T* src = base + (page[i] < 0 ? 0 : page[i] * page_step + (int64_t)((j0 + r) & mask) * token_step);
    if (lane * 4 < p.d) put4(dst + r * ld + lane * 4, src + lane * 4, page[i] >= 0);
  }
}

template <int TR>
struct Smem {
  static size_t bytes(int d) { return (size_t)((16 * TR + 2 * BN) * (d + 4) + 16 * TR * LDP) * sizeof(float); }
};

template <typename T, int TR>
__global__ void __launch_bounds__(NT) paged_simt_kernel(PagedParams p, Scratch s, int tile_tokens) {
  constexpr int BM = 16 * TR;
  extern __shared__ __align__(16) float smem[];
  __shared__ PlanSmem plan_sm;
  __shared__ int again[BM];
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, lane = tid & 31, warp = tid >> 5;
  const int ld = p.d + 4;
  float *Q = smem, *K = Q + BM * ld, *V = K + BN * ld, *P = V + BN * ld;
  tc::grid_dep_launch();
  Walk<BN> w;
  const bool work = plan<BN, NT>(p, tile_tokens, plan_sm, w);
  if (tid == 0) s.shared[blockIdx.x].req = -1;
  if (!work) return;
  const float s2 = p.scale * kLog2e;
  while (w.left > 0) {
    const int n = w.step();
    const Request rq = w.r;
    const T* kp = static_cast<const T*>(p.k) + w.head * p.k_head;
    const T* vp = static_cast<const T*>(p.v) + w.head * p.v_head;
    const int first = (w.span.lo / BN + w.at) * BN;  // first key of the first unit
    for (int r = tid; r < BM; r += NT) again[r] = 0;
    if (tid == 0 && w.at == 0 && n < w.units)
      s.shared[blockIdx.x] = Shared{w.req, w.head, w.tile, w.last_cta()};
    for (int r = warp; r < BM; r += NT / 32) {
      const Row x = row_of(p, rq, w.head, w.tile, tile_tokens, r);
      const T* q = static_cast<const T*>(p.q) + (x.live ? (int64_t)(rq.q0 + x.t) * p.q_stride + (int64_t)x.h * p.d : 0);
      if (lane * 4 < p.d) put4(Q + r * ld + lane * 4, q + lane * 4, x.live);
    }
    load_tile(p, K, ld, kp, p.k_page, p.k_token, w.req, first, w.span);
    cp_commit();
    load_tile(p, V, ld, vp, p.v_page, p.v_token, w.req, first, w.span);
    cp_commit();
    float o[TR][8], m[TR], l[TR];
    int lo[TR], hi[TR];  // keys that the rows see
#pragma unroll
    for (int i = 0; i < TR; ++i) {
#pragma unroll
      for (int c = 0; c < 8; ++c) o[i][c] = 0.f;
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
      const Row x = row_of(p, rq, w.head, w.tile, tile_tokens, ty * TR + i);
      const int pos = rq.kv - rq.len + x.t;
      hi[i] = x.live ? pos + 1 : 0;
      lo[i] = p.window ? max(0, pos - p.window + 1) : 0;
    }
    for (int u = 0; u < n; ++u) {
      const int j0 = first + u * BN;
      cp_wait<1>();
      __syncthreads();
      float a[TR][4];
#pragma unroll
      for (int i = 0; i < TR; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) a[i][j] = 0.f;
#pragma unroll 2
      for (int x = 0; x < p.d; x += 4) {
        float4 kk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4*>(K + (tx + 16 * j) * ld + x);
#pragma unroll
        for (int i = 0; i < TR; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(Q + (ty * TR + i) * ld + x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a[i][j] = fmaf(q.x, kk[j].x, a[i][j]);
            a[i][j] = fmaf(q.y, kk[j].y, a[i][j]);
            a[i][j] = fmaf(q.z, kk[j].z, a[i][j]);
            a[i][j] = fmaf(q.w, kk[j].w, a[i][j]);
          }
        }
      }
      __syncthreads();
      if (u + 1 < n) load_tile(p, K, ld, kp, p.k_page, p.k_token, w.req, j0 + BN, w.span);
      cp_commit();
#pragma unroll
      for (int i = 0; i < TR; ++i) {
        float top = -CUDART_INF_F;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = j0 + tx + 16 * j;
          a[i][j] = key >= lo[i] && key < hi[i] ? a[i][j] * s2 : -CUDART_INF_F;
          top = fmaxf(top, a[i][j]);
        }
#pragma unroll
        for (int x = 8; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float m_new = fmaxf(m[i], top), ref = m_new == -CUDART_INF_F ? 0.f : m_new;
        const float shrink = exp2f(m[i] - ref);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2f(a[i][j] - ref);
          P[(ty * TR + i) * LDP + tx + 16 * j] = e;
          sum += e;
        }
#pragma unroll
        for (int x = 8; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l[i] = fmaf(l[i], shrink, sum);
        m[i] = m_new;
#pragma unroll
        for (int c = 0; c < 8; ++c) o[i][c] *= shrink;
      }
      cp_wait<1>();
      __syncthreads();
      const bool second = 64 + tx * 4 < p.d, one = tx * 4 < p.d;
#pragma unroll 2
      for (int x = 0; x < BN; x += 4) {
        float4 pr[TR];
#pragma unroll
        for (int i = 0; i < TR; ++i) pr[i] = *reinterpret_cast<const float4*>(P + (ty * TR + i) * LDP + x);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          float4 v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
          if (one) v0 = *reinterpret_cast<const float4*>(V + (x + y) * ld + tx * 4);
          if (second) v1 = *reinterpret_cast<const float4*>(V + (x + y) * ld + 64 + tx * 4);
#pragma unroll
          for (int i = 0; i < TR; ++i) {
            const float e = y == 0 ? pr[i].x : y == 1 ? pr[i].y : y == 2 ? pr[i].z : pr[i].w;
            o[i][0] = fmaf(e, v0.x, o[i][0]);
            o[i][1] = fmaf(e, v0.y, o[i][1]);
            o[i][2] = fmaf(e, v0.z, o[i][2]);
            o[i][3] = fmaf(e, v0.w, o[i][3]);
            o[i][4] = fmaf(e, v1.x, o[i][4]);
            o[i][5] = fmaf(e, v1.y, o[i][5]);
            o[i][6] = fmaf(e, v1.z, o[i][6]);
            o[i][7] = fmaf(e, v1.w, o[i][7]);
          }
        }
      }
      __syncthreads();
      if (u + 1 < n) load_tile(p, V, ld, vp, p.v_page, p.v_token, w.req, j0 + BN, w.span);
      cp_commit();
    }
    cp_wait<0>();
    // rows out: whole items to O and lse, parts of items to scratch
    const bool whole = n == w.units;
    const size_t slot = (size_t)(w.at ? 2 * blockIdx.x : 2 * blockIdx.x + 1) * BM;
#pragma unroll
    for (int i = 0; i < TR; ++i) {
      const int r = ty * TR + i;
      const Row x = row_of(p, rq, w.head, w.tile, tile_tokens, r);
      if (!x.live) continue;
      const bool sees = whole ? hi[i] > 0 : l[i] != 0.f;
      const float f = row_factor(l[i], sees);
      bool fine = true;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        o[i][c] = sees ? o[i][c] * f : 0.f;
        fine = fine && fabsf(o[i][c]) <= 3.402823466e38f;
      }
      const size_t out = (size_t)(rq.q0 + x.t) * p.h_q + x.h;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = 64 * j + tx * 4;
        if (c >= p.d) continue;
        const float4 v = {o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
        if (!whole) {
          *reinterpret_cast<float4*>(s.rows + (slot + r) * p.d + c) = v;
        } else if (sizeof(T) == 4) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.O) + out * p.d + c) = v;
        } else {
          __nv_bfloat162 y = __floats2bfloat162_rn(v.x, v.y), z = __floats2bfloat162_rn(v.z, v.w);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + out * p.d + c) =
              uint2{*reinterpret_cast<uint32_t*>(&y), *reinterpret_cast<uint32_t*>(&z)};
        }
      }
      if (tx == 0) {
        if (!whole) s.stat[slot + r] = float2{m[i], l[i]};
        else if (p.lse) p.lse[out] = row_lse(m[i], l[i], sees);
      }
      if (!fine && worth_again(l[i])) again[r] = 1;  // (any of the row's threads)
    }
    __syncthreads();
    for (int r = warp; r < BM; r += NT / 32)
      if (again[r])
        redo_row<T>(p, s, rq, w.req, w.head, row_of(p, rq, w.head, w.tile, tile_tokens, r), first, first + n * BN, whole, slot + r);
    __syncthreads();
    w.advance(p, tile_tokens, n);
  }
}

// Rows of a tile: 16 where a request's rows fit (short windows: two CTAs an SM), 64, 128 otherwise (its thread
// tile of 8 rows x 4 keys takes half as much shared memory traffic for a product as 4 x 4).
struct Shape {
  int tr, ctas;
};
Shape shape_of(const PagedParams& p) {
  const long long rows = (long long)p.max_q * p.group;
  return rows <= 16 ? Shape{1, 2} : rows <= 64 ? Shape{4, 1} : Shape{8, 1};
}

template <typename T, int TR>
cudaError_t launch(const PagedParams& p, const Scratch& s, int G, int tile_tokens, cudaStream_t stream) {
  const size_t bytes = Smem<TR>::bytes(p.d);
  const cudaError_t e = cudaFuncSetAttribute(paged_simt_kernel<T, TR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  paged_simt_kernel<T, TR><<<G, NT, bytes, stream>>>(p, s, tile_tokens);
  return cudaGetLastError();
}

}  // namespace

cudaError_t simt_workspace(const PagedParams& p, int bf16, size_t* bytes) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  const Shape sh = shape_of(p);
  *bytes = scratch_bytes(sms * sh.ctas, 16 * sh.tr, p.d);
  return e;
}

cudaError_t launch_simt(const PagedParams& p, int bf16, void* workspace, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const Shape sh = shape_of(p);
  const int G = sms * sh.ctas, BM = 16 * sh.tr, tile_tokens = BM / p.group;
  const Scratch s = scratch_at(workspace, G, BM, p.d);
  if (bf16)
    e = sh.tr == 1   ? launch<__nv_bfloat16, 1>(p, s, G, tile_tokens, stream)
        : sh.tr == 4 ? launch<__nv_bfloat16, 4>(p, s, G, tile_tokens, stream)
                     : launch<__nv_bfloat16, 8>(p, s, G, tile_tokens, stream);
  else
    e = sh.tr == 1   ? launch<float, 1>(p, s, G, tile_tokens, stream)
        : sh.tr == 4 ? launch<float, 4>(p, s, G, tile_tokens, stream)
                     : launch<float, 8>(p, s, G, tile_tokens, stream);
  return e != cudaSuccess ? e : launch_join(p, bf16, s, G, BM, tile_tokens, stream);
}

}  // namespace paged
}  // namespace gdn
