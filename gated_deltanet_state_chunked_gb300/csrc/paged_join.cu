// gdn_paged_attn: choice of the kernel, scratch, and the joining of partial results (see paged_work.cuh).
#include "paged_work.cuh"

namespace gdn {
namespace paged {
namespace {

// o = sum_c (w_c / sum w) o_c, w_c = l_c 2^(m_c - max m), in the order of the keys: R rows to a warp, 32 / R of their pieces'
// statistics in one load, eight partial rows under way at a time.  Bound by the chain of loads (item, statistics, rows), so
// tiles of 256 rows with few pieces take four rows to a warp (one: 26 us beside 152 shared tiles), tiles of 16 one.
template <typename T, int R>
__global__ void __launch_bounds__(256, 3) paged_join_kernel(PagedParams p, Scratch s, int BM, int tile_tokens) {
  constexpr int P = 32 / R, kAhead = 8 / R;
  tc::grid_dep_wait();
  const Shared sh = s.shared[blockIdx.x];
  if (sh.req < 0) return;
  const int lane = threadIdx.x & 31, row0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * R;
  if (row0 >= min(tile_tokens, sh.r.len - sh.tile * tile_tokens) * p.group) return;
  const int c0 = blockIdx.x, n = sh.last - c0 + 1;
  auto slot = [&](int k) { return (size_t)(k ? 2 * (c0 + k) : 2 * c0 + 1) * BM + row0; };
  // this lane's row of the statistics, and its first piece
  const int my_row = lane / P, my_piece = lane % P;
  auto stat_of = [&](int k) { return k < n && row0 + my_row < BM ? s.stat[slot(k) + my_row] : float2{-CUDART_INF_F, 0.f}; };
  const float2 first = stat_of(my_piece);
  float top = first.x, l = 0.f;
  for (int k = my_piece + P; k < n; k += P) top = fmaxf(top, stat_of(k).x);
#pragma unroll
  for (int o = P / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top == -CUDART_INF_F ? 0.f : top;
  l = first.y * exp2f(first.x - ref);
  for (int k = my_piece + P; k < n; k += P) {
    const float2 st = stat_of(k);
    l += st.y * exp2f(st.x - ref);
  }
#pragma unroll
  for (int o = P / 2; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  // (the weights are divided, not the sum: that could be past fp32)
  const int d4 = p.d / 4;
  const float f = row_factor(l, row_of(p, sh.r, sh.head, sh.tile, tile_tokens, row0 + my_row).t + sh.r.kv - sh.r.len >= 0);
  float4 acc[R];
#pragma unroll
  for (int i = 0; i < R; ++i) acc[i] = float4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < n; k0 += P) {
    const float2 st = k0 ? stat_of(k0 + my_piece) : first;
    const float mine = st.y * exp2f(st.x - ref) * f;
    for (int k = 0; k < min(P, n - k0); k += kAhead) {
      float4 v[kAhead][R];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r)
          v[i][r] = lane < d4 && k0 + k + i < n && row0 + r < BM
                        ? reinterpret_cast<const float4*>(s.rows + (slot(k0 + k + i) + r) * p.d)[lane]
                        : float4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float w = __shfl_sync(0xffffffffu, mine, r * P + ((k + i) & (P - 1)));
          acc[r].x = fmaf(w, v[i][r].x, acc[r].x);
          acc[r].y = fmaf(w, v[i][r].y, acc[r].y);
          acc[r].z = fmaf(w, v[i][r].z, acc[r].z);
          acc[r].w = fmaf(w, v[i][r].w, acc[r].w);
        }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const Row x = row_of(p, sh.r, sh.head, sh.tile, tile_tokens, row0 + r);
    const float sum = __shfl_sync(0xffffffffu, l, r * P), most = __shfl_sync(0xffffffffu, top, r * P);
    if (!x.live) continue;
    const size_t out = (size_t)(sh.r.q0 + x.t) * p.h_q + x.h;
    if (lane < d4) {
      if (sizeof(T) == 4) {
        reinterpret_cast<float4*>(static_cast<float*>(p.O) + out * p.d)[lane] = acc[r];
      } else {
        __nv_bfloat162 a = __floats2bfloat162_rn(acc[r].x, acc[r].y), b = __floats2bfloat162_rn(acc[r].z, acc[r].w);
        reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + out * p.d)[lane] =
            uint2{*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b)};
      }
    }
    if (p.lse && lane == 0) p.lse[out] = row_lse(most, sum, sh.r.kv - sh.r.len + x.t >= 0);
  }
}

template <typename T, int R>
cudaError_t join(const PagedParams& p, const Scratch& s, int G, int BM, int tile_tokens, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(G, (min(BM, tile_tokens * p.group) + 8 * R - 1) / (8 * R));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<T, R>, p, s, BM, tile_tokens);
}

}  // namespace

cudaError_t launch_join(const PagedParams& p, int bf16, const Scratch& s, int G, int BM, int tile_tokens, cudaStream_t stream) {
  if (BM > 32)
    return bf16 ? join<__nv_bfloat16, 4>(p, s, G, BM, tile_tokens, stream) : join<float, 4>(p, s, G, BM, tile_tokens, stream);
  return bf16 ? join<__nv_bfloat16, 1>(p, s, G, BM, tile_tokens, stream) : join<float, 1>(p, s, G, BM, tile_tokens, stream);
}

}  // namespace paged

namespace {

// bf16: up to 16 rows a key head leave 128-row products nearly empty, and are bound by bytes under way (paged_split.cu);
// more go to the tensor pipe (paged_tc.cu).  Pages that have no tensor map (fewer than 8 tokens, strides that it does not
// take): up to 32 rows as before, more on the CUDA cores, as fp32 is (paged_simt.cu).
enum Path { kSplit, kTensor, kCores };
Path path_of(const PagedParams& p, int bf16) {
  const long long rows = (long long)p.max_q * p.group;
  if (!bf16) return kCores;
  return rows <= 16 ? kSplit : paged::tc_supported(p) ? kTensor : rows <= 32 ? kSplit : kCores;
}

}  // namespace

cudaError_t paged_workspace_bytes(const PagedParams& p, int bf16, size_t* bytes) {
  const Path path = path_of(p, bf16);
  return path == kSplit ? paged::split_workspace(p, bytes) : path == kTensor ? paged::tc_workspace(p, bytes) : paged::simt_workspace(p, bf16, bytes);
}
cudaError_t launch_paged_attn(const PagedParams& p, int bf16, void* workspace, cudaStream_t stream) {
  const Path path = path_of(p, bf16);
  return path == kSplit    ? paged::launch_split(p, workspace, stream)
         : path == kTensor ? paged::launch_tc(p, workspace, stream)
                           : paged::launch_simt(p, bf16, workspace, stream);
}

}  // namespace gdn
