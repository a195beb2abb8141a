// gdn_paged_attn, bf16, up to 16 query rows a key head (32 where the pages have no tensor map): single tokens and
// short windows.
//
// Bound by HBM: every key and value is read once for few rows.  So the products are small (warp-level
// mma.sync, 16 rows x 16 keys; tcgen05 tiles of 128 rows would be nearly empty: 128 tokens over up to 16K keys 1,057 us
// on them) and what counts is bytes under way: each warp has a ring of five half stages (16 keys, then their 16 values) of
// its own that runs ahead across items, without any barrier in the loop; two CTAs of four warps an SM keep 128 KB in
// flight and cover each other's ends of items.  Measured: those 128 tokens 610 us, 6.5 TB/s.  Two 16-row tiles a warp
// are bound by the warps' instructions: 64 windows of 20 rows 304 us, on the tcgen05 kernel 167.
// A unit is 64 keys, 16 a warp.  Every warp carries its own maximum, sum and output rows; at an item's end they are
// put together through shared memory, each warp finishing a quarter of the columns.
#include "paged_work.cuh"

namespace gdn {
namespace paged {
namespace {

constexpr int NW = 4, NT = 32 * NW, BN = 16 * NW, kRing = 5;
constexpr int COST = 2;  // of an item, in units (3.5 us against 1.4; with 4: 128 tokens 626 us against 610)

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
__device__ __forceinline__ void ldm4_trans(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
// 16 x 8 += 16 x 16 times 16 x 8
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// DP: head dims up to 64 or 128 (columns behind d are zeros that no load touches); MT: 16-row tiles.
template <int DP, int MT>
struct Lay {
  static constexpr uint32_t kHalf = 16 * DP * 2;  // 16 rows
  static constexpr uint32_t kRows = NW * kRing * kHalf;                  // outputs on their way between warps
  static constexpr uint32_t kStat = kRows + NW * 16 * (DP - DP / NW) * 4;
  static constexpr uint32_t kAgain = kStat + NW * 16 * MT * 8;
  static constexpr uint32_t kPlanAt = kAgain + 16 * MT * 4;
  static constexpr uint32_t kSmem = kPlanAt + sizeof(PlanSmem);
};

template <int DP, int MT>
__global__ void __launch_bounds__(NT, 2) paged_split_kernel(const PagedParams p, const Scratch s, const int tile_tokens) {
  using L = Lay<DP, MT>;
  constexpr int kChunks = DP / 8, kPerLoad = 32 / kChunks;  // 16-byte chunks of a row, rows of one load instruction
  constexpr int kOwn = DP / NW;                             // columns that a warp finishes
  extern __shared__ __align__(128) unsigned char sm[];
  float2* stat = reinterpret_cast<float2*>(sm + L::kStat);
  int* again = reinterpret_cast<int*>(sm + L::kAgain);
  PlanSmem& plan_sm = *reinterpret_cast<PlanSmem*>(sm + L::kPlanAt);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = tc::smem_u32(sm) + warp * kRing * L::kHalf;
  tc::grid_dep_launch();
  if (tid == 0) s.shared[blockIdx.x].req = -1;
  if (p.d < DP)  // columns that no load touches
    for (uint32_t i = tid * 16; i < L::kRows; i += NT * 16) *reinterpret_cast<uint4*>(sm + i) = make_uint4(0u, 0u, 0u, 0u);
  Walk<BN, COST> w;
  if (!plan<BN, COST, NT>(p, tile_tokens, plan_sm, w)) return;
  __syncthreads();

  // ---- loads: a walk of their own, kRing halves ahead
  Walk<BN, COST> lw = w;
  int lu = 0, ln = lw.step(), slot = 0;
  bool values = false;
  const int mask = (1 << p.page_shift) - 1, chunk = lane % kChunks, sub = lane / kChunks;
  int lj = 0, page = -1;  // this lane's key (row lane % 16 of the warp's 16) and its page
  auto look_up = [&]() {
    lj = ((lw.span.lo / BN + lw.at + lu) * BN) + 16 * warp + (lane & 15);
    page = lj >= lw.span.lo && lj < lw.span.hi ? page_of(p, lw.req, lj) : -1;
  };
  look_up();
  auto load_half = [&]() {
    if (lw.left > 0) {
      const __nv_bfloat16* base = values ? static_cast<const __nv_bfloat16*>(p.v) + lw.head * p.v_head
                                         : static_cast<const __nv_bfloat16*>(p.k) + lw.head * p.k_head;
      const int64_t off = page < 0 ? -1 : values ? page * p.v_page + (lj & mask) * p.v_token
                                                 : page * p.k_page + (lj & mask) * p.k_token;
      const uint32_t dst = ring + slot * L::kHalf;
      if (__all_sync(0xffffffffu, page >= 0)) {
#pragma unroll
        for (int i = 0; i < 16 / kPerLoad; ++i) {
          const int row = kPerLoad * i + sub;
          const int64_t at = __shfl_sync(0xffffffffu, off, row);
          if (8 * chunk < p.d) cp16(dst + row * (2 * DP) + ((chunk ^ (row & 7)) << 4), base + at + 8 * chunk);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16 / kPerLoad; ++i) {
          const int row = kPerLoad * i + sub;
          const int64_t at = __shfl_sync(0xffffffffu, off, row);
          if (8 * chunk < p.d)
            cp16_or_zero(dst + row * (2 * DP) + ((chunk ^ (row & 7)) << 4), base + (at < 0 ? 0 : at + 8 * chunk), at >= 0);
        }
      }
      if (values) {
        if (++lu == ln) {
          lw.advance(p, tile_tokens, ln);
          lu = 0;
          ln = lw.step();
        }
        if (lw.left > 0) look_up();
      }
      values = !values;
    }
    cp_commit();
    slot = slot + 1 == kRing ? 0 : slot + 1;
  };
#pragma unroll 1
  for (int i = 0; i < kRing; ++i) load_half();

  const float s2 = p.scale == 0.f ? 1e-37f : p.scale * kLog2e;  // (for 0 a factor that still takes -inf to -inf)
  const float masked = s2 > 0.f ? -CUDART_INF_F : CUDART_INF_F;
  int at_half = 0;  // ring place of the next half to use
  while (w.left > 0) {
    const int n = w.step();
    const Request rq = w.r;
    const int first = (w.span.lo / BN + w.at) * BN;
    uint32_t q[MT][DP / 16][4];
    float o[MT][DP / 8][4], ref[MT][2], l[MT][2];
    int lo[MT][2], hi[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Row x = row_of(p, rq, w.head, w.tile, tile_tokens, 16 * t + 8 * i + lane / 4);
        const int pos = rq.kv - rq.len + x.t;
        // (a row that is none sees everything, so that it calls for no masking; nothing of it is stored)
        hi[t][i] = x.live ? pos + 1 : INT_MAX;
        lo[t][i] = x.live ? low_of(p, pos) : 0;
        ref[t][i] = -CUDART_INF_F;
        l[t][i] = 0.f;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)(rq.q0 + x.t) * p.q_stride + (int64_t)x.h * p.d;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int c = 16 * k + 8 * j + 2 * (lane & 3);
            q[t][k][i + 2 * j] = x.live && c < p.d ? *reinterpret_cast<const uint32_t*>(src + c) : 0u;
          }
#pragma unroll
        for (int c = 0; c < DP / 8; ++c) o[t][c][2 * i] = o[t][c][2 * i + 1] = 0.f;
      }
    for (int u = 0; u < n; ++u) {
      const int j0 = first + u * BN + 16 * warp;
      // scores of 16 keys
      float sc[MT][2][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[t][j][e] = 0.f;
      cp_wait<kRing - 1>();
      __syncwarp();
      {
        const int row = (lane & 7) + 8 * (lane >> 4);
        const uint32_t kt = ring + at_half * L::kHalf + row * (2 * DP);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          uint32_t b[4];
          ldm4(kt + (((2 * k + ((lane >> 3) & 1)) ^ (row & 7)) << 4), b);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            mma(sc[t][0], q[t][k], b[0], b[1]);
            mma(sc[t][1], q[t][k], b[2], b[3]);
          }
        }
      }
      __syncwarp();
      load_half();
      at_half = at_half + 1 == kRing ? 0 : at_half + 1;
      uint32_t pr[MT][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (__any_sync(0xffffffffu, lo[t][0] > j0 || hi[t][0] < j0 + 16 || lo[t][1] > j0 || hi[t][1] < j0 + 16)) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = j0 + 8 * j + 2 * (lane & 3) + (e & 1);
              sc[t][j][e] = key >= lo[t][e >> 1] && key < hi[t][e >> 1] ? sc[t][j][e] : masked;
            }
        }
        float m[2];
        bool grown = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) sc[t][j][2 * i + e] *= s2;
          m[i] = fmaxf(fmaxf(sc[t][0][2 * i], sc[t][0][2 * i + 1]), fmaxf(sc[t][1][2 * i], sc[t][1][2 * i + 1]));
          m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
          m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 2));
          grown = grown || m[i] > ref[t][i] + 8.f;
        }
        if (__any_sync(0xffffffffu, grown)) {  // (a row's reference follows its maximum by steps of more than 8)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float next = fmaxf(ref[t][i], m[i]);
            const float f = ref[t][i] == -CUDART_INF_F ? 0.f : exp2_fast(ref[t][i] - next);
            ref[t][i] = next;
            l[t][i] *= f;
#pragma unroll
            for (int c = 0; c < DP / 8; ++c) {
              o[t][c][2 * i] *= f;
              o[t][c][2 * i + 1] *= f;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float r = ref[t][i] == -CUDART_INF_F ? 0.f : ref[t][i];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float e0 = exp2_fast(sc[t][j][2 * i] - r), e1 = exp2_fast(sc[t][j][2 * i + 1] - r);
            l[t][i] += e0 + e1;
            pr[t][i + 2 * j] = pack_bf16(e0, e1);
          }
        }
      }
      cp_wait<kRing - 1>();
      __syncwarp();
      {
        const int row = lane & 15;
        const uint32_t vt = ring + at_half * L::kHalf + row * (2 * DP);
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
          uint32_t b[4];
          ldm4_trans(vt + (((2 * c + (lane >> 4)) ^ (row & 7)) << 4), b);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            mma(o[t][2 * c], pr[t], b[0], b[1]);
            mma(o[t][2 * c + 1], pr[t], b[2], b[3]);
          }
        }
      }
      __syncwarp();
      load_half();
      at_half = at_half + 1 == kRing ? 0 : at_half + 1;
    }
    // ---- the item's end
    const bool whole = n == w.units;
    if (tid == 0 && w.at == 0 && !whole)
      s.shared[blockIdx.x] = Shared{w.req, w.head, w.tile, w.last_cta(), rq, 0};
    const size_t slot_row = (size_t)(w.at ? 2 * blockIdx.x : 2 * blockIdx.x + 1) * (16 * MT);
    if (tid < 16 * MT) again[tid] = 0;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 1);
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 2);
        if ((lane & 3) == 0) stat[warp * 16 * MT + 16 * t + 8 * i + lane / 4] = float2{ref[t][i], l[t][i]};
      }
    float* rows = reinterpret_cast<float*>(sm + L::kRows);
    const int me = lane / 4, col = 2 * (lane & 3);
    constexpr int kTiles = kOwn / 8;  // 8-column tiles that a warp finishes
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      // to each other warp its columns: [to][from, in order][16 rows][kOwn]
#pragma unroll
      for (int c = 0; c < DP / 8; ++c) {
        const int to = c / kTiles;
        if (to == warp) continue;
        float* dst = rows + ((to * (NW - 1) + (warp < to ? warp : warp - 1)) * 16) * kOwn + 8 * (c % kTiles) + col;
        *reinterpret_cast<float2*>(dst + me * kOwn) = float2{o[t][c][0], o[t][c][1]};
        *reinterpret_cast<float2*>(dst + (me + 8) * kOwn) = float2{o[t][c][2], o[t][c][3]};
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * t + 8 * i + me;
        float2 st[NW];
        float top = -CUDART_INF_F;
#pragma unroll
        for (int x = 0; x < NW; ++x) {
          st[x] = stat[x * 16 * MT + r];
          top = fmaxf(top, st[x].x);
        }
        const float base = top == -CUDART_INF_F ? 0.f : top;
        float sum = 0.f, f[NW];
#pragma unroll
        for (int x = 0; x < NW; ++x) {
          f[x] = exp2_fast(st[x].x - base);
          sum = fmaf(st[x].y, f[x], sum);
        }
        const bool sees = whole ? hi[t][i] > 0 : sum != 0.f;
        const float norm = row_factor(sum, sees);
        const Row x = row_of(p, rq, w.head, w.tile, tile_tokens, r);
        const size_t out = (size_t)(rq.q0 + x.t) * p.h_q + x.h;
        bool fine = true;
#pragma unroll
        for (int c = 0; c < kTiles; ++c) {
          const int cc = kOwn * warp + 8 * c + col;
          float y0 = 0.f, y1 = 0.f;
#pragma unroll
          for (int from = 0; from < NW; ++from) {  // (in the order of the warps, whoever adds)
            const float g = f[from] * norm;
            float2 v;
            if (from == warp) {
              v = float2{0.f, 0.f};
#pragma unroll
              for (int z = 0; z < NW; ++z)  // (the warp's own columns, by a fixed register index)
                if (z == warp) v = float2{o[t][z * kTiles + c][2 * i], o[t][z * kTiles + c][2 * i + 1]};
            } else {
              v = *reinterpret_cast<const float2*>(rows + ((warp * (NW - 1) + (from < warp ? from : from - 1)) * 16 + 8 * i + me) * kOwn +
                                                   8 * c + col);
            }
            y0 = fmaf(g, v.x, y0);
            y1 = fmaf(g, v.y, y1);
          }
          if (!sees) y0 = y1 = 0.f;
          if (cc < p.d && x.live) {
            fine = fine && fabsf(y0) <= 3.402823466e38f && fabsf(y1) <= 3.402823466e38f;
            if (whole) *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.O) + out * p.d + cc) = pack_bf16(y0, y1);
            else *reinterpret_cast<float2*>(s.rows + (slot_row + r) * p.d + cc) = float2{y0, y1};
          }
        }
        if (x.live && warp == 0 && (lane & 3) == 0) {
          if (!whole) s.stat[slot_row + r] = float2{top, sum};
          else if (p.lse) p.lse[out] = row_lse(top, sum, sees);
        }
        if (!fine && worth_again(sum)) again[r] = 1;
      }
      __syncthreads();
    }
    for (int r = warp; r < 16 * MT; r += NW)
      if (again[r])
        redo_row<__nv_bfloat16>(p, s, rq, w.req, w.head, row_of(p, rq, w.head, w.tile, tile_tokens, r), first, first + n * BN, whole,
                                slot_row + r);
    w.advance(p, tile_tokens, n);
    __syncthreads();  // (the flags are read before they are cleared)
  }
  cp_wait<0>();
}

template <int DP, int MT>
cudaError_t launch(const PagedParams& p, const Scratch& s, int G, int tile_tokens, cudaStream_t stream) {
  constexpr size_t bytes = Lay<DP, MT>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(paged_split_kernel<DP, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  paged_split_kernel<DP, MT><<<G, NT, bytes, stream>>>(p, s, tile_tokens);
  return cudaGetLastError();
}

int rows_of(const PagedParams& p) { return (long long)p.max_q * p.group <= 16 ? 16 : 32; }

}  // namespace

cudaError_t split_workspace(const PagedParams& p, size_t* bytes) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  *bytes = scratch_bytes(2 * sms, rows_of(p), p.d);
  return e;
}

cudaError_t launch_split(const PagedParams& p, void* workspace, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int G = 2 * sms, BM = rows_of(p), tile_tokens = BM / p.group;
  const Scratch s = scratch_at(workspace, G, BM, p.d);
  if (p.d <= 64)
    e = BM == 16 ? launch<64, 1>(p, s, G, tile_tokens, stream) : launch<64, 2>(p, s, G, tile_tokens, stream);
  else
    e = BM == 16 ? launch<128, 1>(p, s, G, tile_tokens, stream) : launch<128, 2>(p, s, G, tile_tokens, stream);
  return e != cudaSuccess ? e : launch_join(p, 1, s, G, BM, tile_tokens, stream);
}

}  // namespace paged
}  // namespace gdn
