// gdn_paged_attn, bf16, on the tensor cores (tcgen05 + TMEM): windows and chunks.
//
// A tile is 256 query rows (tokens x the query heads of one key head), as two halves of 128 that take turns on
// the tensor pipe, against units of 128 keys (paged_work.cuh deals the units out).  Per unit and half, all with
// M = 128 and fp32 accumulators in TMEM:
//   S = Q K^T    A = Q, B = K, both K-major in shared memory
//   O += P V     A = P, bf16, in TMEM in the place of S; B = V, [key][d] as it lies in the cache (MN-major)
// With p = 2^(s - r), s = scale log2(e) q.k, a row's reference r follows its running maximum only when that has grown
// by more than 8 (P stays below 2^8, O and the sum of weights below 2^8 times what they would be): the first units
// of an item rescale O, few others do.
// P is rounded to bf16, as O itself is: its roundings are independent, so O's error grows from 1.7e-3 (its own) to
// 2.4e-3; the sum of weights and lse take the unrounded ones.
//
// Warps: 0-3 and 4-7 the rows of the two halves, a thread a row: maximum, exponentials, P, and at the end O out; 8-11 load
// Q, K and V, 32 rows of a tile each; 12 issues the MMAs.  Keys and values pass through a ring of five 32 KB stages.
// Units inside a request come by tensor copies, a page (up to 32 rows of it) at a time; the first and last
// unit of a request, pages of fewer than 8 tokens and strides that a tensor map does not take by cp.async, which fills
// the places of keys that nobody sees with zeros (what lies there may be no number).  With cp.async alone the loading
// warps bound the kernel (1,700 clocks to issue a stage: chunk of 2048 at 32K 1,173 us).
// Registers are moved from the loading and issuing warps to the rows'.  Every hand-off is an mbarrier; every wait
// is bounded.
#include <atomic>

#include "paged_work.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace paged {
namespace {

using namespace tc;
using tcp::kWaitNs;

constexpr int NT = 512, BM = 256, BN = 128, kStages = 5, kLag = 3;
constexpr int kRegsLaunch = 128, kRegsRows = 184, kRegsLoad = 80, kRegsIssue = 64;
static_assert(2 * kRegsRows + kRegsLoad + kRegsIssue <= 4 * kRegsLaunch, "what a launch holds");
// A stage that is waited for may be kLag loads away from the one being issued, and the issuing warp holds a stage of
// values until it has multiplied the next keys.
static_assert(kStages >= kLag + 2, "stages");
constexpr uint32_t kTile = 32768, kAtom = 16384;  // 128 rows x 128 bf16: two swizzled atoms of 64 columns
constexpr uint32_t kQ = 0, kRing = 2 * kTile, kBarAt = kRing + kStages * kTile, kMisc = kBarAt + 256, kPlanAt = kMisc + 16,
                   kSmem = kPlanAt + sizeof(PlanSmem);
static_assert(kSmem <= 232448, "shared memory");
constexpr uint32_t cS = 0, cO = 256;  // TMEM columns of the halves' S (and P) and O, 128 each
constexpr uint64_t kLongNs = 2 * kWaitNs;  // waits that rows computed again may hold up

enum Bar { kFull = 0, kEmpty = kFull + kStages, kQFull = kEmpty + kStages, kQEmpty, kS, kP = kS + 2, kO = kP + 2, kOFree = kO + 2,
           kDrain = kOFree + 2, kBars };
static_assert(kBars * 8 <= 256, "barrier area");

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows of a tile's second half: none for short windows.
__device__ __forceinline__ bool second_half(const PagedParams& p, const Request& r, int tile, int tile_tokens) {
  return min(tile_tokens, r.len - tile * tile_tokens) * p.group > 128;
}

// A tensor map of the key or value pages: d, then tokens, heads and pages by ascending stride, at these places.
struct PageMap {
  int token, head, page;  // 1 to 3
  int rows;               // tokens of a box; 0: no map
};
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, const PageMap& m, uint64_t* bar, int x, int token,
                                              int head, int page) {
  const int c1 = m.token == 1 ? token : m.head == 1 ? head : page, c2 = m.token == 2 ? token : m.head == 2 ? head : page,
            c3 = m.token == 3 ? token : m.head == 3 ? head : page;
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__global__ void __launch_bounds__(NT, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const PageMap mk,
                    const PageMap mv, const PagedParams p, const Scratch s, const int tile_tokens) {
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + kBarAt);
  volatile int* dead = reinterpret_cast<int*>(sm + kMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kMisc) + 1;
  PlanSmem& plan_sm = *reinterpret_cast<PlanSmem*>(sm + kPlanAt);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = warp >> 2, quad = warp & 3;

  if (smem_u32(sm) & 1023u) {  // (the swizzled tiles could not be addressed)
    if (tid == 0) {
      s.shared[blockIdx.x].req = -1;
      atomicExch(p.status, GDN_ERR_CUDA);
    }
    return;
  }
  grid_dep_launch();
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int b = 0; b < kBars; ++b) {
      int count = 1;
      if ((b >= kFull && b < kFull + kStages) || b == kQFull || (b >= kP && b < kP + 2) || (b >= kOFree && b < kOFree + 2)) count = 4;
      mbar_init(&bar[b], count);
    }
    mbar_fence_init();
    *dead = 0;
    s.shared[blockIdx.x].req = -1;
  }
  Walk<BN> w;
  const bool work = plan<BN, NT>(p, tile_tokens, plan_sm, w);
  if (!work) w.left = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](int b, int phase, uint64_t limit = kWaitNs) {
    if (mbar_wait(&bar[b], (uint32_t)(phase & 1), limit)) return true;
    *dead = 1;
    return false;
  };
  auto arrive = [&](int b) {  // one arrival per warp, behind what its threads did before
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[b]);
  };
  // Every role walks the same items; stages, tiles and items are counted by each for itself, and the phases go by
  // these counts.  A barrier is never two completions ahead of a waiter: what completes it next follows from what the
  // waiter does after the wait.

  if (group < 2) {
    // ------------------------------------------------------------ rows
    regs_inc<kRegsRows>();
    const uint32_t at = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t at_s = at + cS + 128 * group, at_o = at + cO + 128 * group;
    // scores in log2 units; for a scale of 0 (every key weighs the same) a factor that still takes -inf to -inf
    const float s2 = p.scale == 0.f ? 1e-37f : p.scale * kLog2e;
    const float masked = s2 > 0.f ? -CUDART_INF_F : CUDART_INF_F;
    const int r = 128 * group + 32 * quad + lane;
    int done = 0;  // units of this half
    bool ok = true;
    while (w.left > 0 && ok) {
      const int n = w.step();
      const Request rq = w.r;
      if (group == 0 || second_half(p, rq, w.tile, tile_tokens)) {
        const int first = (w.span.lo / BN + w.at) * BN;
        const Row x = row_of(p, rq, w.head, w.tile, tile_tokens, r);
        const int pos = rq.kv - rq.len + x.t;
        // (a row that is none sees everything, so that it calls for no masking; nothing of it is stored)
        const int hi = x.live ? pos + 1 : INT_MAX, lo = x.live && p.window ? max(0, pos - p.window + 1) : 0;
        float ref = -CUDART_INF_F, l = 0.f;
        for (int u = 0; u < n; ++u, ++done) {
          if (!(ok = wait(kS + group, done))) break;
          tc_fence_after();
          float a[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(at_s + 32 * i, a[i]);
          tmem_ld_wait();
          const int j0 = first + u * BN;
          if (__any_sync(0xffffffffu, lo > j0 || hi < j0 + BN)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // bits lo - j .. hi - j - 1 of the 32 columns
              const int from = max(0, lo - j0 - 32 * i), to = min(32, max(0, hi - j0 - 32 * i));
              const uint32_t seen = from >= to ? 0u : (0xffffffffu << from) & (0xffffffffu >> (32 - to));
#pragma unroll
              for (int j = 0; j < 32; ++j) a[i][j] = (seen >> j) & 1u ? a[i][j] : masked;
            }
          }
          float top[4];
          if (s2 > 0.f) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              top[i] = a[i][0];
#pragma unroll
              for (int j = 1; j < 32; ++j) top[i] = fmaxf(top[i], a[i][j]);
            }
            top[0] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              top[i] = a[i][0];
#pragma unroll
              for (int j = 1; j < 32; ++j) top[i] = fminf(top[i], a[i][j]);
            }
            top[0] = fminf(fminf(top[0], top[1]), fminf(top[2], top[3]));
          }
          const float m = top[0] * s2;
          const bool grown = m > ref + 8.f;  // (-inf + 8 too)
          if (__any_sync(0xffffffffu, grown)) {
            const float f = grown ? (ref == -CUDART_INF_F ? 0.f : exp2_fast(ref - m)) : 1.f;
            if (grown) ref = m;
            l *= f;
            if (u > 0) {
              if (!(ok = wait(kO + group, done - 1))) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < p.d; c += 32) {
                float o[32];
                tmem_ld32(at_o + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] *= f;
                tmem_st32(at_o + c, o);
              }
              tmem_st_wait();
            }
          }
          const float neg = ref == -CUDART_INF_F ? 0.f : -ref;
          const uint64_t s2s2 = pair(s2, s2), nn = pair(neg, neg);
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float e0, e1;
              unpair(fma2(pair(a[i][j], a[i][j + 1]), s2s2, nn), e0, e1);
              e0 = exp2_fast(e0);
              e1 = exp2_fast(e1);
              sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], pair(e0, e1));
              o[j / 2] = pack_bf16(e0, e1);
            }
            tmem_st16(at_s + 16 * i, o);
          }
          float y0, y1;
          unpair(add2(sum[0], sum[1]), y0, y1);
          l += y0 + y1;
          tmem_st_wait();
          tc_fence_before();
          arrive(kP + group);
        }
        if (!ok) break;
        if (!(ok = wait(kO + group, done - 1))) break;
        tc_fence_after();
        // rows out: whole items to O and lse, parts of items to scratch
        const bool whole = n == w.units;
        const bool sees = whole ? hi > 0 : l != 0.f;
        const float f = row_factor(l, sees);
        const size_t slot_row = (size_t)(w.at ? 2 * blockIdx.x : 2 * blockIdx.x + 1) * BM + r;
        const size_t out = (size_t)(rq.q0 + x.t) * p.h_q + x.h;
        bool fine = true;
        // (16 columns at a time: an item's end runs through this code once, and what it costs is fetching the code.  Wider
        // steps that store 64 bytes of a row at once: 10,000 clocks of an item, 38,000 the first time)
#pragma unroll 1
        for (int c = 0; c < p.d; c += 16) {
          float o[16];
          tmem_ld16(at_o + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[j] = sees ? o[j] * f : 0.f;
            fine = fine && fabsf(o[j]) <= 3.402823466e38f;  // (columns behind d are zeros times weights, or like the others)
          }
          if (x.live) {
#pragma unroll
            for (int j = 0; j < 16; j += 8)
              if (c + j < p.d) {
                if (whole) {
                  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.O) + out * p.d + c + j) =
                      make_uint4(pack_bf16(o[j], o[j + 1]), pack_bf16(o[j + 2], o[j + 3]), pack_bf16(o[j + 4], o[j + 5]),
                                 pack_bf16(o[j + 6], o[j + 7]));
                } else {
                  float4* to = reinterpret_cast<float4*>(s.rows + slot_row * p.d + c + j);
                  to[0] = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                  to[1] = make_float4(o[j + 4], o[j + 5], o[j + 6], o[j + 7]);
                }
              }
          }
        }
        tc_fence_before();
        arrive(kOFree + group);
        if (x.live) {
          if (!whole) s.stat[slot_row] = float2{ref, l};
          else if (p.lse) p.lse[out] = row_lse(ref, l, sees);
        }
        unsigned again = __ballot_sync(0xffffffffu, x.live && !fine && worth_again(l));
        __syncwarp();
        for (; again; again &= again - 1) {
          const int rr = __ffs(again) - 1;
          redo_row<__nv_bfloat16>(p, s, rq, w.req, w.head, row_of(p, rq, w.head, w.tile, tile_tokens, r - lane + rr), first,
                                  first + n * BN, whole, slot_row - lane + rr);
        }
      }
      if (tid == 0 && w.at == 0 && n < w.units)
        s.shared[blockIdx.x] = Shared{w.req, w.head, w.tile, w.cta_of(w.pos + w.units - 1)};
      w.advance(p, tile_tokens, n);
    }
  } else if (group == 2) {
    // ------------------------------------------------------------ loads
    regs_dec<kRegsLoad>();
    const uint32_t base = smem_u32(sm);
    const int mask = (1 << p.page_shift) - 1, chunk = lane & 7, sub = lane >> 3;
    const int wide = (p.d + 15) / 16 * 16;  // columns that the products cover
    int pend[kLag], issued = 0, items = 0;
#pragma unroll
    for (int i = 0; i < kLag; ++i) pend[i] = -1;
    bool ok = true;
    // A load is announced kLag loads later, when this thread's part has landed (generic writes, which the MMAs
    // read through the async proxy).
    auto push = [&](int b) {
      cp_commit();
      if (pend[0] >= 0) {
        cp_wait<kLag>();
        fence_async_smem();
        arrive(pend[0]);
      }
#pragma unroll
      for (int i = 0; i + 1 < kLag; ++i) pend[i] = pend[i + 1];
      pend[kLag - 1] = b;
    };
    auto flush = [&]() {
      cp_wait<0>();
      fence_async_smem();
#pragma unroll
      for (int i = 0; i < kLag; ++i) {
        if (pend[i] >= 0) arrive(pend[i]);
        pend[i] = -1;
      }
    };
    // 32 rows of a 128-row tile, eight lanes to 128 bytes of a row; off: lane's own row's offset, or -1
    auto load_rows = [&](uint32_t tile, const __nv_bfloat16* src, int64_t off) {
#pragma unroll 4
      for (int i = 0; i < 8; ++i) {
        const int64_t at = __shfl_sync(0xffffffffu, off, 4 * i + sub);
        const int row = 32 * quad + 4 * i + sub;
        const uint32_t dst = tile + row * 128 + ((chunk ^ (row & 7)) << 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = 64 * half + 8 * chunk;
          if (c < wide) {
            const bool there = at >= 0 && c < p.d;
            cp16(dst + half * kAtom, src + (there ? at + c : 0), there);
          }
        }
      }
    };
    while (w.left > 0 && ok) {
      const int n = w.step();
      const int first = (w.span.lo / BN + w.at) * BN;
      flush();
      if (items > 0 && !(ok = wait(kQEmpty, items - 1, kLongNs))) break;
      const int halves = second_half(p, w.r, w.tile, tile_tokens) ? 2 : 1;
      for (int half = 0; half < halves; ++half) {
        const Row x = row_of(p, w.r, w.head, w.tile, tile_tokens, 128 * half + 32 * quad + lane);
        load_rows(base + kQ + half * kTile, static_cast<const __nv_bfloat16*>(p.q),
                  x.live ? (int64_t)(w.r.q0 + x.t) * p.q_stride + (int64_t)x.h * p.d : -1);
      }
      push(kQFull);
      const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(p.k) + w.head * p.k_head;
      const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(p.v) + w.head * p.v_head;
      const Span span = w.span;
      auto page_at = [&](int u) {
        const int j = first + u * BN + 32 * quad + lane;
        return u < n && j >= span.lo && j < span.hi ? page_of(p, w.req, j) : -1;
      };
      // A stage by tensor copies: each warp's 32 rows are a part of one page, or several whole ones.
      const int atoms = p.d > 64 ? 2 : 1;
      auto copy_rows = [&](const CUtensorMap* map, const PageMap& m, int st, int j, int page) {
        const int boxes = 32 / m.rows;
        if (lane == 0) mbar_arrive_expect_tx(&bar[kFull + st], 32u * 128u * atoms);
        __syncwarp();
        if (lane < boxes * atoms) {
          const int box = lane & (boxes - 1), atom = lane / boxes;
          tma_load_page(base + kRing + st * kTile + atom * kAtom + (32 * quad + box * m.rows) * 128, map, m, &bar[kFull + st], 64 * atom,
                        (j + box * m.rows) & mask, w.head, page);
        }
        __syncwarp();
      };
      auto next_stage = [&](int& st) {
        st = issued % kStages;
        return issued < kStages || (ok = wait(kEmpty + st, issued / kStages - 1, kLongNs));
      };
      const bool maps = mk.rows > 0 && mv.rows > 0;
      int page = page_at(0);
      for (int u = 0; u < n; ++u) {
        const int j0 = first + u * BN, j = j0 + 32 * quad;
        int st;
        if (maps && j0 >= span.lo && j0 + BN <= span.hi) {
          // (the box's page, from the lane of its first key; a page outside the cache reads as zeros)
          int kb = __shfl_sync(0xffffffffu, page, (lane & (32 / mk.rows - 1)) * mk.rows);
          int vb = __shfl_sync(0xffffffffu, page, (lane & (32 / mv.rows - 1)) * mv.rows);
          kb = kb < 0 ? p.n_pages : kb;
          vb = vb < 0 ? p.n_pages : vb;
          if (!next_stage(st)) break;
          copy_rows(&map_k, mk, st, j, kb);
          ++issued;
          page = page_at(u + 1);
          if (!next_stage(st)) break;
          copy_rows(&map_v, mv, st, j, vb);
          ++issued;
          if (u == 0) flush();  // (the queries, which nothing else pushes on)
        } else {
          const int64_t token = (j + lane) & mask;
          const int64_t k_off = page < 0 ? -1 : page * p.k_page + token * p.k_token;
          const int64_t v_off = page < 0 ? -1 : page * p.v_page + token * p.v_token;
          if (!next_stage(st)) break;
          load_rows(base + kRing + st * kTile, kp, k_off);
          push(kFull + st);
          ++issued;
          page = page_at(u + 1);
          if (!next_stage(st)) break;
          load_rows(base + kRing + st * kTile, vp, v_off);
          push(kFull + st);
          ++issued;
          if (maps) flush();  // (nothing pushes these on while tensor copies follow)
        }
      }
      if (!ok) break;
      ++items;
      w.advance(p, tile_tokens, n);
    }
    flush();
    if (!ok)  // let this warp's tensor copies in flight land (their stages may lack other warps' arrivals: briefly)
      for (int i = max(0, issued - kStages); i < issued; ++i)
        mbar_wait(&bar[kFull + i % kStages], (uint32_t)((i / kStages) & 1), kWaitNs / 100);
  } else {
    regs_dec<kRegsIssue>();
    if (quad == 0) {
      // ---------------------------------------------------------- MMAs
      const int nk = (p.d + 15) / 16;
      const uint32_t idQK = idesc_bf16(128, 128, false, false), idPV = idesc_bf16(128, 16 * nk, false, true);
      const uint64_t dQ = sdesc_sw128(smem_u32(sm + kQ), 16, 1024), dK = sdesc_sw128(smem_u32(sm + kRing), 16, 1024),
                     dV = sdesc_sw128(smem_u32(sm + kRing), kAtom, 1024);
      auto qk = [&](int half, int st) {
        if (elect_one()) {
          const uint64_t q = dQ + (uint64_t)((half * kTile) >> 4), k = dK + (uint64_t)((st * kTile) >> 4);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < nk) {
              const uint64_t off = (uint64_t)(((i >> 2) * kAtom + (i & 3) * 32) >> 4);
              mma_bf16(tmem + cS + 128 * half, q + off, k + off, idQK, i > 0);
            }
          mma_commit(&bar[kS + half]);
        }
        __syncwarp();
      };
      auto pv = [&](int half, int st, bool add) {
        if (elect_one()) {
          const uint64_t v = dV + (uint64_t)((st * kTile) >> 4);
#pragma unroll
          for (int i = 0; i < BN / 16; ++i)
            mma_bf16_ts(tmem + cO + 128 * half, tmem + cS + 128 * half + 8 * i, v + (uint64_t)((i * 2048) >> 4), idPV, add || i > 0);
          mma_commit(&bar[kO + half]);
        }
        __syncwarp();
      };
      auto commit = [&](int b) {
        if (elect_one()) mma_commit(&bar[b]);
        __syncwarp();
      };
      int g = 0, items = 0;           // stages taken, items
      int units[2] = {0, 0}, outs[2] = {0, 0};  // units and items of the halves
      bool ok = true;
      while (w.left > 0 && ok) {
        const int n = w.step(), halves = second_half(p, w.r, w.tile, tile_tokens) ? 2 : 1;
        if (!(ok = wait(kQFull, items, kLongNs)) || !(ok = wait(kFull + g % kStages, g / kStages))) break;
        tc_fence_after();
        for (int half = 0; half < halves; ++half) qk(half, g % kStages);
        commit(kEmpty + g % kStages);
        if (n == 1) commit(kQEmpty);
        ++g;
        for (int u = 0; u < n && ok; ++u) {
          const int st_v = g % kStages, st_k = (g + 1) % kStages;
          if (!(ok = wait(kFull + st_v, g / kStages))) break;
          for (int half = 0; half < halves; ++half) {
            if (!(ok = wait(kP + half, units[half], kLongNs))) break;
            if (u == 0 && outs[half] > 0 && !(ok = wait(kOFree + half, outs[half] - 1, kLongNs))) break;
            tc_fence_after();
            pv(half, st_v, u > 0);
            ++units[half];
            if (u + 1 < n) {
              if (half == 0 && !(ok = wait(kFull + st_k, (g + 1) / kStages))) break;
              tc_fence_after();
              qk(half, st_k);
            }
          }
          if (!ok) break;
          commit(kEmpty + st_v);
          if (u + 1 < n) commit(kEmpty + st_k);
          if (u + 2 == n) commit(kQEmpty);
          g += u + 1 < n ? 2 : 1;
        }
        for (int half = 0; half < halves; ++half) ++outs[half];
        ++items;
        w.advance(p, tile_tokens, n);
      }
      if (elect_one()) mma_commit(&bar[kDrain]);
      __syncwarp();
      mbar_wait(&bar[kDrain], 0, kWaitNs);
    }
  }
  tc_fence_before();
  __syncthreads();
  // (a wait that gave up: the loads have landed and the MMAs are done, each by its own warps; the results are unspecified)
  if (*dead && tid == 0) atomicExch(p.status, GDN_ERR_TIMEOUT);
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// The kernel is launched with the registers that the warpgroups' shares add up to (with fewer, a warpgroup
// that asks for more would wait): checked once.
cudaError_t check_registers() {
  static std::atomic<bool> checked{false};
  if (checked.load(std::memory_order_acquire)) return cudaSuccess;
  cudaFuncAttributes have;
  const cudaError_t e = cudaFuncGetAttributes(&have, reinterpret_cast<const void*>(paged_tc_kernel));
  if (e != cudaSuccess) return e;
  if (have.numRegs != kRegsLaunch) return cudaErrorInvalidKernelImage;
  checked.store(true, std::memory_order_release);
  return cudaSuccess;
}

// The map of pages with these strides; its `rows` stay 0 where there is none.
void make_page_map(CUtensorMap* map, PageMap* m, const PagedParams& p, const void* base, int64_t page, int64_t token, int64_t head) {
  *m = PageMap{1, 2, 3, 0};
  auto enc = encode_fn();
  const int size = 1 << p.page_shift, rows = size < 32 ? size : 32;
  if (!enc || rows < 8) return;  // (a box starts at a multiple of 8 rows of the swizzled tile)
  struct Dim {
    int64_t stride;
    int64_t size;
    int box;
    int* at;
  } dims[3] = {{token, size, rows, &m->token}, {head, p.h_kv, 1, &m->head}, {page, p.n_pages, 1, &m->page}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j + 1 < 3; ++j)
      if (dims[j].stride > dims[j + 1].stride) {
        const Dim x = dims[j];
        dims[j] = dims[j + 1];
        dims[j + 1] = x;
      }
  cuuint64_t sizes[4] = {(cuuint64_t)p.d, 0, 0, 0}, strides[3];
  cuuint32_t box[4] = {64, 0, 0, 0}, es[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    if (dims[i].stride == 0 && dims[i].size > 1) return;
    *dims[i].at = i + 1;
    sizes[i + 1] = (cuuint64_t)dims[i].size;
    strides[i] = (cuuint64_t)(dims[i].stride > 0 ? dims[i].stride * 2 : 16);
    box[i + 1] = (cuuint32_t)dims[i].box;
  }
  if (enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), sizes, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
    m->rows = rows;
}

}  // namespace

cudaError_t tc_workspace(const PagedParams& p, size_t* bytes) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  *bytes = scratch_bytes(sms, BM, p.d);
  return e;
}

cudaError_t launch_tc(const PagedParams& p, void* workspace, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e == cudaSuccess) e = check_registers();
  // (in each call: the attribute belongs to the current context)
  if (e == cudaSuccess) e = cudaFuncSetAttribute(paged_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  const int tile_tokens = BM / p.group;
  const Scratch s = scratch_at(workspace, sms, BM, p.d);
  CUtensorMap map_k{}, map_v{};
  PageMap mk, mv;
  make_page_map(&map_k, &mk, p, p.k, p.k_page, p.k_token, p.k_head);
  make_page_map(&map_v, &mv, p, p.v, p.v_page, p.v_token, p.v_head);
  paged_tc_kernel<<<sms, NT, kSmem, stream>>>(map_k, map_v, mk, mv, p, s, tile_tokens);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join(p, 1, s, sms, BM, tile_tokens, stream);
}

}  // namespace paged
}  // namespace gdn
