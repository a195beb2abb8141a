// gdn_paged_attn: choice of the kernel, scratch, and the joining of partial results (see paged_work.cuh).
#include "paged_work.cuh"

namespace gdn {
namespace paged {
namespace {

// o = sum_c (w_c / sum w) o_c, w_c = l_c 2^(m_c - max m): one warp a row, its pieces in the order of the
// keys.  The statistics are read side by side, then the rows eight at a time: two trips to L2 for most items.
template <typename T>
__global__ void __launch_bounds__(256, 3) paged_join_kernel(PagedParams p, Scratch s, int BM, int tile_tokens) {
  tc::grid_dep_wait();
  const Shared sh = s.shared[blockIdx.x];
  if (sh.req < 0) return;
  const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5);
  bool bad;
  const Request rq = request_of(p, sh.req, INT_MIN, &bad);
  if (row >= BM) return;
  const Row x = row_of(p, rq, sh.head, sh.tile, tile_tokens, row);
  if (!x.live) return;
  const bool sees = rq.kv - rq.len + x.t >= 0;
  const int c0 = blockIdx.x, n = sh.last - c0 + 1;
  auto slot = [&](int k) { return (size_t)(k ? 2 * (c0 + k) : 2 * c0 + 1) * BM + row; };
  float top = -CUDART_INF_F, l = 0.f;
  for (int k = lane; k < n; k += 32) top = fmaxf(top, s.stat[slot(k)].x);
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top == -CUDART_INF_F ? 0.f : top;
  for (int k = lane; k < n; k += 32) {
    const float2 st = s.stat[slot(k)];
    l += st.y * exp2f(st.x - ref);
  }
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float f = row_factor(l, sees);  // (the weights are divided, not the sum: that could be past fp32)
  const int d4 = p.d / 4;
  float4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < n; k0 += 32) {
    float w_mine = 0.f;
    if (k0 + lane < n) {
      const float2 st = s.stat[slot(k0 + lane)];
      w_mine = st.y * exp2f(st.x - ref) * f;
    }
    // (eight rows under way at a time)
    constexpr int kAhead = 8;
    for (int k = 0; k < min(32, n - k0); k += kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        v[i] = lane < d4 && k0 + k + i < n ? reinterpret_cast<const float4*>(s.rows + slot(k0 + k + i) * p.d)[lane]
                                           : float4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float w = __shfl_sync(0xffffffffu, w_mine, k + i);
        acc.x = fmaf(w, v[i].x, acc.x);
        acc.y = fmaf(w, v[i].y, acc.y);
        acc.z = fmaf(w, v[i].z, acc.z);
        acc.w = fmaf(w, v[i].w, acc.w);
      }
    }
  }
  const size_t out = (size_t)(rq.q0 + x.t) * p.h_q + x.h;
  if (lane < d4) {
    if (sizeof(T) == 4) {
      reinterpret_cast<float4*>(static_cast<float*>(p.O) + out * p.d)[lane] = acc;
    } else {
      __nv_bfloat162 a = __floats2bfloat162_rn(acc.x, acc.y), b = __floats2bfloat162_rn(acc.z, acc.w);
      uint2 u = {*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b)};
      reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + out * p.d)[lane] = u;
    }
  }
  if (p.lse && lane == 0) p.lse[out] = row_lse(top, l, sees);
}

}  // namespace

cudaError_t launch_join(const PagedParams& p, int bf16, const Scratch& s, int G, int BM, int tile_tokens, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(G, (min(BM, tile_tokens * p.group) + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, paged_join_kernel<__nv_bfloat16>, p, s, BM, tile_tokens)
              : cudaLaunchKernelEx(&cfg, paged_join_kernel<float>, p, s, BM, tile_tokens);
}

}  // namespace paged

// bf16: up to 16 rows a key head (single tokens) leave 128-row products nearly empty and need bytes under way; pages that have no tensor
// map (fewer than 8 tokens, strides that it does not take) fall to the CUDA cores, as fp32 does.
cudaError_t paged_workspace_bytes(const PagedParams& p, int bf16, size_t* bytes) {
  if (bf16 && paged::split_supported(p)) return paged::split_workspace(p, bytes);
  if (bf16 && paged::tc_supported(p)) return paged::tc_workspace(p, bytes);
  return paged::simt_workspace(p, bf16, bytes);
}
cudaError_t launch_paged_attn(const PagedParams& p, int bf16, void* workspace, cudaStream_t stream) {
  if (bf16 && paged::split_supported(p)) return paged::launch_split(p, workspace, stream);
  if (bf16 && paged::tc_supported(p)) return paged::launch_tc(p, workspace, stream);
  return paged::launch_simt(p, bf16, workspace, stream);
}

}  // namespace gdn
