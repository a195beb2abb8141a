// gdn_paged_attn on the CUDA cores.
#include "paged_work.cuh"

namespace gdn {
namespace paged {
namespace {

// One CTA of 256 threads, tiles of BM = 16 TR query rows x 64 keys.  Thread (ty, tx) = (tid / 16, tid % 16)
// holds rows TR ty .. and keys tx + 16 j of the scores, columns 2 tx + 32 j (and the next) of the outputs, as pairs for the
// packed FMAs (two products in one instruction; the scores' pairs are even and odd places of the head).  Keys and values
// each have one buffer: the next tile's keys arrive while the values are multiplied, its values while the scores are.
// Bound by the FMA pipe in long chunks (1,024 tokens over 3,000, 32 heads of 128, fp32: 1.53 ms, 38 TFLOP/s); short ones by
// their few units on each CTA.  Single tokens (64 over up to 6,000 keys: 540 us, 3 TB/s) by shared memory, for which 16-row
// tiles with few rows are wide: warps without rows only load (with all of them at work 914 us).
constexpr int NT = 256, BN = 64, LDP = BN + 4;
constexpr int COST = 0;  // (of an item, in units: a unit takes 13 us, the rest of an item 4)

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
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
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
__global__ void __launch_bounds__(NT, TR <= 2 ? 2 : 1) paged_simt_kernel(PagedParams p, Scratch s, int tile_tokens) {
  constexpr int BM = 16 * TR;
  extern __shared__ __align__(16) float smem[];
  __shared__ PlanSmem plan_sm;
  __shared__ int again[BM];
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, lane = tid & 31, warp = tid >> 5;
  const int ld = p.d + 4;
  float *Q = smem, *K = Q + BM * ld, *V = K + BN * ld, *P = V + BN * ld;
  tc::grid_dep_launch();
  Walk<BN, COST> w;
  const bool work = plan<BN, COST, NT>(p, tile_tokens, plan_sm, w);
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
      s.shared[blockIdx.x] = Shared{w.req, w.head, w.tile, w.last_cta(), rq, 0};
    for (int r = warp; r < BM; r += NT / 32) {
      const Row x = row_of(p, rq, w.head, w.tile, tile_tokens, r);
      const T* q = static_cast<const T*>(p.q) + (x.live ? (int64_t)(rq.q0 + x.t) * p.q_stride + (int64_t)x.h * p.d : 0);
      if (lane * 4 < p.d) put4(Q + r * ld + lane * 4, q + lane * 4, x.live);
    }
    load_tile(p, K, ld, kp, p.k_page, p.k_token, w.req, first, w.span);
    cp_commit();
    load_tile(p, V, ld, vp, p.v_page, p.v_token, w.req, first, w.span);
    cp_commit();
    uint64_t o[TR][4];
    float m[TR], l[TR];
    int lo[TR], hi[TR];  // keys that the rows see
#pragma unroll
    for (int i = 0; i < TR; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0ull;
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
      const Row x = row_of(p, rq, w.head, w.tile, tile_tokens, ty * TR + i);
      const int pos = rq.kv - rq.len + x.t;
      hi[i] = x.live ? pos + 1 : 0;
      lo[i] = low_of(p, pos);
    }
    int any = 0;
#pragma unroll
    for (int i = 0; i < TR; ++i) any |= hi[i] > 0;
    const bool busy = __any_sync(0xffffffffu, any);  // (a warp whose rows are none, or see nothing, has only loads to do)
    for (int u = 0; u < n; ++u) {
      const int j0 = first + u * BN;
      cp_wait<1>();
      __syncthreads();
      float a[TR][4];
      if (busy) {
        uint64_t acc[TR][4];
#pragma unroll
        for (int i = 0; i < TR; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
#pragma unroll 2
        for (int x = 0; x < p.d; x += 4) {
          ulonglong2 kk[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const ulonglong2*>(K + (tx + 16 * j) * ld + x);
#pragma unroll
          for (int i = 0; i < TR; ++i) {
            const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(Q + (ty * TR + i) * ld + x);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fma2(q.y, kk[j].y, fma2(q.x, kk[j].x, acc[i][j]));
          }
        }
#pragma unroll
        for (int i = 0; i < TR; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 y = unpair(acc[i][j]);
            a[i][j] = y.x + y.y;
          }
      }
      __syncthreads();
      if (u + 1 < n) load_tile(p, K, ld, kp, p.k_page, p.k_token, w.req, j0 + BN, w.span);
      cp_commit();
      if (busy) {
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
          const uint64_t ss = pair(shrink, shrink);
#pragma unroll
          for (int c = 0; c < 4; ++c) o[i][c] = mul2(o[i][c], ss);
        }
      }
      cp_wait<1>();
      __syncthreads();
      const int cols = (p.d + 31) / 32;  // (places behind d in the last columns: what the buffer holds there, not stored)
#pragma unroll 1
      for (int x = 0; x < (busy ? BN : 0); x += 4) {
        float4 pr[TR];
#pragma unroll
        for (int i = 0; i < TR; ++i) pr[i] = *reinterpret_cast<const float4*>(P + (ty * TR + i) * LDP + x);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < cols) {
            uint64_t v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) v[y] = *reinterpret_cast<const uint64_t*>(V + (x + y) * ld + 32 * j + 2 * tx);
#pragma unroll
            for (int i = 0; i < TR; ++i) {
              o[i][j] = fma2(pair(pr[i].x, pr[i].x), v[0], o[i][j]);
              o[i][j] = fma2(pair(pr[i].y, pr[i].y), v[1], o[i][j]);
              o[i][j] = fma2(pair(pr[i].z, pr[i].z), v[2], o[i][j]);
              o[i][j] = fma2(pair(pr[i].w, pr[i].w), v[3], o[i][j]);
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
      const size_t out = (size_t)(rq.q0 + x.t) * p.h_q + x.h;
      bool fine = true;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = 32 * j + 2 * tx;
        if (c >= p.d) continue;
        float2 v = unpair(o[i][j]);
        v = sees ? float2{v.x * f, v.y * f} : float2{0.f, 0.f};
        fine = fine && fabsf(v.x) <= 3.402823466e38f && fabsf(v.y) <= 3.402823466e38f;
        if (!whole) {
          *reinterpret_cast<float2*>(s.rows + (slot + r) * p.d + c) = v;
        } else if (sizeof(T) == 4) {
          *reinterpret_cast<float2*>(static_cast<float*>(p.O) + out * p.d + c) = v;
        } else {
          *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.O) + out * p.d + c) = __floats2bfloat162_rn(v.x, v.y);
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

// Rows of a tile: the fewest of 16, 32, 64 and 128 that hold a request's (the thread tile of 8 rows x 4 keys takes half as
// much shared memory traffic for a product as 4 x 4); up to 32 two CTAs an SM fit, whose loads cover each other's work.
struct Shape {
  int tr, ctas;
};
Shape shape_of(const PagedParams& p) {
  const long long rows = (long long)p.max_q * p.group;
  return rows <= 16 ? Shape{1, 2} : rows <= 32 ? Shape{2, 2} : rows <= 64 ? Shape{4, 1} : Shape{8, 1};
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
  auto run = [&](auto t) {
    using T = decltype(t);
    return sh.tr == 1   ? launch<T, 1>(p, s, G, tile_tokens, stream)
           : sh.tr == 2 ? launch<T, 2>(p, s, G, tile_tokens, stream)
           : sh.tr == 4 ? launch<T, 4>(p, s, G, tile_tokens, stream)
                        : launch<T, 8>(p, s, G, tile_tokens, stream);
  };
  e = bf16 ? run(__nv_bfloat16()) : run(0.f);
  return e != cudaSuccess ? e : launch_join(p, bf16, s, G, BM, tile_tokens, stream);
}

}  // namespace paged
}  // namespace gdn
