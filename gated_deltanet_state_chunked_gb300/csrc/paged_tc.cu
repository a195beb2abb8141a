// gdn_paged_attn, bf16, on the tensor cores (tcgen05 + TMEM + TMA): windows and chunks.
//
// A tile is up to 256 query rows (tokens x the query heads of one key head) against units of 128 keys (paged_work.cuh
// deals the units out).  Two halves take turns on the tensor pipe: rows 0-127 and 128-255 of a tile, or, of a tile of up to 128
// rows, the even and the odd units.  Per unit and half, all with M = 128 and fp32 accumulators in TMEM:
//   S = Q K^T    A = Q, B = K, both K-major in shared memory
//   O += P V     A = P, bf16, in TMEM in the place of S; B = V, [key][d] as it lies in the cache (MN-major)
// With p = 2^(s - r), s = scale log2(e) q.k, a row's reference r follows its running maximum only when that has grown
// by more than 8 (P stays below 2^8, O and the sum of weights below 2^8 times what they would be): the first units
// of an item rescale O, few others do.
// P is rounded to bf16, as O itself is: its roundings are independent, so O's error grows from 1.7e-3 (its own) to
// 2.4e-3; the sum of weights and lse take the unrounded ones.
//
// Warps: 0-3 and 4-7 the halves' rows, a thread a row: maximum, exponentials, P.  8-11 the outputs: an item's O goes
// from TMEM into registers at once, so that the next item's products can begin, and is stored beside them.  12 issues
// the MMAs.  13 loads Q and K, 14 V, into a ring of five 32 KB stages, by tensor copies (a page at a time, up to 128 rows of it).
// The rows of V behind a request's end (they may hold anything) are cleared before they are handed on.  Registers are
// moved from the last eight warps to the rows'.  Every hand-off is an mbarrier; every wait is bounded.
//
// Bound: in long chunks each half's chain (scores 512 clocks, weights about 1,400, their product with the values 512, three
// hand-offs) while the other half's runs beside it, 3,300 clocks a unit of 256 rows, where the tensor pipe alone would take
// 2,048; S = Q K^T reads shared memory at its limit.  Measured, 32/8 heads of 128: a chunk of 2,048 at the end of 32,768 keys
// 695 us, 1.53 PFLOP/s (753 in a long run, under the board's power limit); 64 windows of 5 over up to 6,005 keys 155 us,
// 5.3 TB/s; 12 ragged chunks of 6,007 tokens, window 1,777, 24/4 heads of 96, 152 us (an item of 15 units costs four more).
// Multiplying P by halves took the first from 732 to 714 us, a warp each for keys and values 16-token pages from 830 to 736.
#include <atomic>

#include "paged_work.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace paged {
namespace {

using namespace tc;
using tcp::kWaitNs;

constexpr int NT = 512, BM = 256, BN = 128, kStages = 5;
constexpr int COST = 4;  // of an item, in units (7 us against 1.75; with 2: chunk of 4096 from nothing 167 us against 151)
constexpr int kRegsLaunch = 128, kRegsRows = 168, kRegsOut = 120, kRegsIssue = 56;
static_assert(2 * kRegsRows + kRegsOut + kRegsIssue <= 4 * kRegsLaunch, "what a launch holds");
constexpr uint32_t kTile = 32768, kAtom = 16384;  // 128 rows x 128 bf16: two swizzled atoms of 64 columns
// Q: two atoms of 256 rows; the ring; the halves' (reference, sum) of each row
constexpr uint32_t kQ = 0, kQAtom = 2 * kAtom, kRing = 2 * kQAtom, kBarAt = kRing + kStages * kTile, kMisc = kBarAt + 256,
                   kStatAt = kMisc + 16, kPlanAt = kStatAt + 2 * 128 * 8, kSmem = kPlanAt + sizeof(PlanSmem);
static_assert(kSmem <= 232448, "shared memory");
constexpr uint32_t cS = 0, cO = 256;  // TMEM columns of the halves' S (and P) and O, 128 each
constexpr uint64_t kLongNs = 8 * kWaitNs;  // waits that rows computed again may hold up

enum Bar { kFull = 0, kEmpty = kFull + kStages, kQFull = kEmpty + kStages, kQEmpty, kTail, kDrain, kS, kP = kS + 2 /* by columns: 0-63, 64-127 */, kO = kP + 4,
           kStat = kO + 2, kOFree = kStat + 2, kBars = kOFree + 2 };
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


// A tensor map of the key or value pages: d, then tokens, heads and pages by ascending stride, at these places.
struct PageMap {
  int token, head, page;  // 1 to 3
  int rows;               // tokens of a box
};
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, const PageMap& m, uint64_t* bar, int x, int token,
                                              int head, int page) {
  const int c1 = m.token == 1 ? token : m.head == 1 ? head : page, c2 = m.token == 2 ? token : m.head == 2 ? head : page,
            c3 = m.token == 3 ? token : m.head == 3 ? head : page;
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Units of an item's n that half h works on: all of them, or (split: a tile of up to 128 rows) every other one.
__device__ __forceinline__ int units_of_half(bool split, int n, int h) { return split ? (n + 1 - h) / 2 : n; }
__device__ __forceinline__ bool split_units(const PagedParams& p, const Request& r, int tile, int tile_tokens) {
  return min(tile_tokens, r.len - tile * tile_tokens) * p.group <= 128;
}

__global__ void __launch_bounds__(NT, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const PageMap mk, const PageMap mv, const PagedParams p, const Scratch s,
                    const int tile_tokens) {
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + kBarAt);
  volatile int* dead = reinterpret_cast<int*>(sm + kMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kMisc) + 1;
  float2* stat = reinterpret_cast<float2*>(sm + kStatAt);
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
    for (int b = 0; b < kBars; ++b)
      mbar_init(&bar[b], (b >= kP && b < kP + 4) || (b >= kStat && b < kOFree + 2) ? 4 : 1);
    mbar_fence_init();
    *dead = 0;
    s.shared[blockIdx.x].req = -1;
  }
  if (warp == 13 && lane < 3) tma_prefetch_desc(lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v);
  Walk<BN, COST> w;
  const bool work = plan<BN, COST, NT>(p, tile_tokens, plan_sm, w);
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
  // Every role walks the same items; stages, the halves' units and items are counted by each for itself, and the phases go
  // by these counts.  A barrier is never two completions ahead of a waiter: what completes it next follows from what the
  // waiter does after the wait.
  const uint32_t at = tmem + ((uint32_t)(32 * quad) << 16);

  if (group < 2) {
    // ------------------------------------------------------------ rows
    regs_inc<kRegsRows>();
    const uint32_t at_s = at + cS + 128 * group, at_o = at + cO + 128 * group;
    // scores in log2 units; for a scale of 0 (every key weighs the same) a factor that still takes -inf to -inf
    const float s2 = p.scale == 0.f ? 1e-37f : p.scale * kLog2e;
    const float masked = s2 > 0.f ? -CUDART_INF_F : CUDART_INF_F;
    int done = 0, items = 0;  // units and items of this half
    bool ok = true;
    while (w.left > 0 && ok) {
      const int n = w.step();
      const bool split = split_units(p, w.r, w.tile, tile_tokens);
      const int mine = units_of_half(split, n, group);
      if (mine > 0) {
        const int first = (w.span.lo / BN + w.at) * BN;
        const Row x = row_of(p, w.r, w.head, w.tile, tile_tokens, (split ? 0 : 128 * group) + 32 * quad + lane);
        const int pos = w.r.kv - w.r.len + x.t;
        // (a row that is none sees everything, so that it calls for no masking; nothing of it is stored)
        const int hi = x.live ? pos + 1 : INT_MAX, lo = x.live ? low_of(p, pos) : 0;
        float ref = -CUDART_INF_F, l = 0.f;
        for (int i_u = 0; i_u < mine; ++i_u, ++done) {
          if (!(ok = wait(kS + group, done, kLongNs))) break;
          tc_fence_after();
          float a[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(at_s + 32 * i, a[i]);
          tmem_ld_wait();
          const int j0 = first + (split ? 2 * i_u + group : i_u) * BN;
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
            if (i_u > 0) {
              if (!(ok = wait(kO + group, done - 1))) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < p.d; c += 16) {
                float o[16];
                tmem_ld16(at_o + c, o);
                tmem_ld_wait();
                uint32_t y[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(o[j] * f);
                tmem_st16(at_o + c, y);
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
            if (i & 1) {  // (half of P is multiplied while the other half is made)
              tmem_st_wait();
              tc_fence_before();
              arrive(kP + group + (i & 2));
            }
          }
          float y0, y1;
          unpair(add2(sum[0], sum[1]), y0, y1);
          l += y0 + y1;
        }
        if (!ok) break;
        if (items > 0 && !(ok = wait(kOFree + group, items - 1, kLongNs))) break;  // (the item before it has been read)
        stat[128 * group + 32 * quad + lane] = float2{ref, l};
        arrive(kStat + group);
        ++items;
      }
      w.advance(p, tile_tokens, n);
    }
  } else if (group == 2) {
    // ------------------------------------------------------------ outputs
    regs_dec<kRegsOut>();
    int done[2] = {0, 0}, items[2] = {0, 0};  // units and items of the halves
    bool ok = true;
    while (w.left > 0 && ok) {
      const int n = w.step();
      const Request rq = w.r;
      const bool split = split_units(p, rq, w.tile, tile_tokens), whole = n == w.units;
      const int first = (w.span.lo / BN + w.at) * BN;
      const size_t slot = (size_t)(w.at ? 2 * blockIdx.x : 2 * blockIdx.x + 1) * BM;
#pragma unroll 1
      for (int h = 0; h < (split ? 1 : 2); ++h) {
        const bool both = split && n > 1;  // (the halves' sums are one row's)
        done[h] += units_of_half(split, n, h);
        if (!(ok = wait(kStat + h, items[h], kLongNs) && wait(kO + h, done[h] - 1))) break;
        ++items[h];
        if (both) {
          done[1] += units_of_half(split, n, 1);
          if (!(ok = wait(kStat + 1, items[1], kLongNs) && wait(kO + 1, done[1] - 1))) break;
          ++items[1];
        }
        tc_fence_after();
        const int r = 128 * h + 32 * quad + lane;
        const Row x = row_of(p, rq, w.head, w.tile, tile_tokens, r);
        const bool sees = rq.kv - rq.len + x.t >= 0;
        float2 st = stat[r];
        float f0 = 1.f, f1 = 0.f;
        if (both) {
          const float2 other = stat[128 + 32 * quad + lane];
          const float top = fmaxf(st.x, other.x), base = top == -CUDART_INF_F ? 0.f : top;
          f0 = exp2_fast(st.x - base);
          f1 = exp2_fast(other.x - base);
          st = float2{top, fmaf(st.y, f0, other.y * f1)};
        }
        // (a part of an item in which the row sees nothing is left as zeros)
        const float norm = (whole ? sees : st.y != 0.f) ? row_factor(st.y, true) : 0.f;
        const bool zero = norm == 0.f;
        f0 *= norm;
        f1 *= norm;
        const size_t out = (size_t)(rq.q0 + x.t) * p.h_q + x.h, slot_row = slot + r;
        const uint32_t at_o = at + cO + 128 * h;
        bool fine = true;
        auto columns = [&](int c, float (&o)[16]) {
          tmem_ld16(at_o + c, o);
          if (both) {
            float y[16];
            tmem_ld16(at_o + 128 + c, y);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = fmaf(o[j], f0, y[j] * f1);
          } else {
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= f0;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[j] = zero ? 0.f : o[j];
            fine = fine && fabsf(o[j]) <= 3.402823466e38f;
          }
        };
        auto release = [&]() {
          tc_fence_before();
          arrive(kOFree + h);
          if (both) arrive(kOFree + 1);
        };
        if (whole) {
          uint32_t y[8][8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (16 * c < p.d) {
              float o[16];
              columns(16 * c, o);
#pragma unroll
              for (int j = 0; j < 8; ++j) y[c][j] = pack_bf16(o[2 * j], o[2 * j + 1]);
            }
          release();
          if (x.live) {
            uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.O) + out * p.d);
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (8 * c < p.d) to[c] = make_uint4(y[c / 2][4 * (c & 1)], y[c / 2][4 * (c & 1) + 1], y[c / 2][4 * (c & 1) + 2], y[c / 2][4 * (c & 1) + 3]);
            if (p.lse) p.lse[out] = row_lse(st.x, st.y, sees);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < p.d; c += 16) {
            float o[16];
            columns(c, o);
            if (x.live) {
              float4* to = reinterpret_cast<float4*>(s.rows + slot_row * p.d + c);
#pragma unroll
              for (int j = 0; j < 16; j += 4)
                if (c + j < p.d) to[j / 4] = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
            }
          }
          release();
          if (x.live) s.stat[slot_row] = st;
        }
        unsigned again = __ballot_sync(0xffffffffu, x.live && !fine && worth_again(st.y));
        __syncwarp();
        for (; again; again &= again - 1) {
          const int rr = __ffs(again) - 1;
          redo_row<__nv_bfloat16>(p, s, rq, w.req, w.head, row_of(p, rq, w.head, w.tile, tile_tokens, r - lane + rr), first,
                                  first + n * BN, whole, slot_row - lane + rr);
        }
      }
      if (tid == 256 && w.at == 0 && !whole)
        s.shared[blockIdx.x] = Shared{w.req, w.head, w.tile, w.last_cta(), rq, 0};
      w.advance(p, tile_tokens, n);
    }
  } else {
    regs_dec<kRegsIssue>();
    if (quad == 0) {
      // ---------------------------------------------------------- MMAs
      const int nk = (p.d + 15) / 16;
      const uint32_t idQK = idesc_bf16(128, 128, false, false), idPV = idesc_bf16(128, 16 * nk, false, true);
      const uint64_t dQ = sdesc_sw128(smem_u32(sm + kQ), 16, 1024), dK = sdesc_sw128(smem_u32(sm + kRing), 16, 1024),
                     dV = sdesc_sw128(smem_u32(sm + kRing), kAtom, 1024);
      // S of half `h` from the rows of half `rows`; then the stage is free, and behind an item's last product Q
      auto qk = [&](int h, int rows, int st, bool free, bool last) {
        if (elect_one()) {
          const uint64_t q = dQ + (uint64_t)((rows * kAtom) >> 4), k = dK + (uint64_t)((st * kTile) >> 4);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < nk)
              mma_bf16(tmem + cS + 128 * h, q + (uint64_t)(((i >> 2) * kQAtom + (i & 3) * 32) >> 4),
                       k + (uint64_t)(((i >> 2) * kAtom + (i & 3) * 32) >> 4), idQK, i > 0);
          mma_commit(&bar[kS + h]);
          if (free) mma_commit(&bar[kEmpty + st]);
          if (last) mma_commit(&bar[kQEmpty]);
        }
        __syncwarp();
      };
      int g = 0, items = 0;                       // stages taken, items
      int units[2] = {0, 0}, outs[2] = {0, 0};    // units and items of the halves
      bool ok = true;
      auto full = [&](int i) { return wait(kFull + i % kStages, i / kStages, kLongNs); };
      // O (+)= P V of the half's next unit, by halves of P as they come; before an item's first, the outputs of the
      // half's item before have been read
      auto pv = [&](int h, int st, bool first, bool free) {
        const uint64_t v = dV + (uint64_t)((st * kTile) >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wait(kP + h + 2 * half, units[h], kLongNs)) return false;
          if (half == 0 && first && outs[h] > 0 && !wait(kOFree + h, outs[h] - 1, kLongNs)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int i = 4 * half; i < 4 * half + 4; ++i)
              mma_bf16_ts(tmem + cO + 128 * h, tmem + cS + 128 * h + 8 * i, v + (uint64_t)((i * 2048) >> 4), idPV, !first || i > 0);
            if (half == 1) {
              mma_commit(&bar[kO + h]);
              if (free) mma_commit(&bar[kEmpty + st]);
            }
          }
          __syncwarp();
        }
        ++units[h];
        return true;
      };
      while (w.left > 0 && ok) {
        const int n = w.step();
        const bool split = split_units(p, w.r, w.tile, tile_tokens);
        if (!(ok = wait(kQFull, items, kLongNs) && full(g))) break;
        tc_fence_after();
        if (split) {
          qk(0, 0, g % kStages, true, n == 1);
          if (n > 1) {
            if (!(ok = full(g + 2))) break;
            tc_fence_after();
            qk(1, 0, (g + 2) % kStages, true, n == 2);
          }
          for (int u = 0; u < n; ++u) {
            const int h = u & 1, sv = g + 2 * u + 1, sk = g + 2 * u + 4;
            if (!(ok = full(sv) && pv(h, sv % kStages, u < 2, true))) break;
            if (u + 2 < n) {
              if (!(ok = full(sk))) break;
              tc_fence_after();
              qk(h, 0, sk % kStages, true, u + 3 == n);
            }
          }
        } else {
          for (int h = 0; h < 2; ++h) qk(h, h, g % kStages, h == 1, h == 1 && n == 1);
          for (int u = 0; u < n && ok; ++u) {
            const int sv = g + 2 * u + 1, sk = g + 2 * u + 2;
            if (!(ok = full(sv))) break;
            for (int h = 0; h < 2; ++h) {
              if (!(ok = pv(h, sv % kStages, u == 0, h == 1))) break;
              if (u + 1 < n) {
                if (h == 0) {
                  if (!(ok = full(sk))) break;
                  tc_fence_after();
                }
                qk(h, h, sk % kStages, h == 1, h == 1 && u + 2 == n);
              }
            }
          }
        }
        for (int h = 0; h < 2; ++h) outs[h] += units_of_half(split, n, h) > 0;
        g += 2 * n;
        ++items;
        w.advance(p, tile_tokens, n);
      }
      if (elect_one()) mma_commit(&bar[kDrain]);
      __syncwarp();
      mbar_wait(&bar[kDrain], 0, kWaitNs);
    } else if (quad < 3) {
      // ---------------------------------------------------------- loads: warp 13 Q and K, warp 14 V
      const uint32_t base = smem_u32(sm);
      const bool values = quad == 2;
      const CUtensorMap* map = values ? &map_v : &map_k;
      const PageMap m = values ? mv : mk;
      const int mask = (1 << p.page_shift) - 1, atoms = p.d > 64 ? 2 : 1;
      const int boxes = BN / m.rows, box = lane & (boxes - 1), atom = lane / boxes;  // this lane's box of a stage
      int g = values ? 1 : 0, items = 0, tails = 0;  // the next stage (every other one), items, tails
      bool ok = true;
      while (w.left > 0 && ok) {
        const int n = w.step(), first = (w.span.lo / BN + w.at) * BN;
        const Span span = w.span;
        // the page of this lane's box of unit u: outside the cache (where a copy reads zeros) if no key of it is wanted
        auto page_at = [&](int u) {
          const int j = first + u * BN + box * m.rows;
          const int page = u < n && j < span.hi && j + m.rows > span.lo ? page_of(p, w.req, j) : -1;
          return page < 0 ? p.n_pages : page;
        };
        int page = page_at(0);
        for (int u = 0; u < n; ++u, g += 2) {
          const int st = g % kStages, live = w.r.kv - (first + u * BN);  // rows of the unit before the request's end
          const bool tail = values && live < BN;
          const int b = tail ? kTail : kFull + st;
          if (g >= kStages && !(ok = wait(kEmpty + st, g / kStages - 1, kLongNs))) break;
          if (lane == 0) mbar_arrive_expect_tx(&bar[b], (uint32_t)BN * 128u * atoms);
          __syncwarp();
          if (lane < boxes * atoms)
            tma_load_page(base + kRing + st * kTile + atom * kAtom + box * m.rows * 128, map, m, &bar[b], 64 * atom,
                          (first + u * BN + box * m.rows) & mask, w.head, page);
          __syncwarp();
          page = page_at(u + 1);
          if (u == 0 && !values) {
            if (items > 0 && !(ok = wait(kQEmpty, items - 1, kLongNs))) break;
            if (lane == 0) mbar_arrive_expect_tx(&bar[kQFull], (uint32_t)(p.group * tile_tokens) * 128u * atoms);
            __syncwarp();
            if (lane < atoms)
              tma_load_3d(base + kQ + lane * kQAtom, &map_q, &bar[kQFull], 64 * lane, w.head * p.group, w.r.q0 + w.tile * tile_tokens);
            __syncwarp();
          }
          if (tail) {
            if (!(ok = wait(kTail, tails++))) break;
            for (int i = max(live, 0) * 8 + lane; i < BN * 8; i += 32)
              for (int a = 0; a < atoms; ++a)
                *reinterpret_cast<uint4*>(sm + kRing + st * kTile + a * kAtom + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
            fence_async_smem();
            arrive(kFull + st);
          }
        }
        if (!ok) break;
        ++items;
        w.advance(p, tile_tokens, n);
      }
      if (!ok) {  // let the copies in flight land
        for (int i = max(values ? 1 : 0, g - 2 * kStages); i < g; i += 2)
          mbar_wait(&bar[kFull + i % kStages], (uint32_t)((i / kStages) & 1), kWaitNs / 100);
        if (!values) mbar_wait(&bar[kQFull], (uint32_t)(items & 1), kWaitNs / 100);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // (a wait that gave up: the loads have landed and the MMAs are done, each by its own warp; the results are unspecified)
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

// The map of pages with these strides.
bool make_page_map(CUtensorMap* map, PageMap* m, const PagedParams& p, const void* base, int64_t page, int64_t token, int64_t head) {
  auto enc = encode_fn();
  const int size = 1 << p.page_shift, rows = size < BN ? size : BN;
  *m = PageMap{1, 2, 3, rows};
  if (!enc) return false;
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
    *dims[i].at = i + 1;
    sizes[i + 1] = (cuuint64_t)dims[i].size;
    strides[i] = (cuuint64_t)(dims[i].stride > 0 ? dims[i].stride * 2 : 16);
    box[i + 1] = (cuuint32_t)dims[i].box;
  }
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), sizes, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int tile_tokens_of(const PagedParams& p) { return p.max_q < BM / p.group ? p.max_q : BM / p.group; }

// Boxes of tile_tokens tokens x the query heads of a key head: rows in the order of a tile.
bool make_query_map(CUtensorMap* map, const PagedParams& p) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t sizes[3] = {(cuuint64_t)p.d, (cuuint64_t)p.h_q, (cuuint64_t)p.total}, strides[2] = {(cuuint64_t)p.d * 2, (cuuint64_t)p.q_stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)tile_tokens_of(p)}, es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), sizes, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap q, k, v;
  PageMap mk, mv;
};
bool make_maps(Maps* m, const PagedParams& p) {
  return make_page_map(&m->k, &m->mk, p, p.k, p.k_page, p.k_token, p.k_head) &&
         make_page_map(&m->v, &m->mv, p, p.v, p.v_page, p.v_token, p.v_head) && make_query_map(&m->q, p);
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
  Maps m{};
  if (e == cudaSuccess && !make_maps(&m, p)) e = cudaErrorInvalidValue;
  if (e == cudaSuccess) e = check_registers();
  // (in each call: the attribute belongs to the current context)
  if (e == cudaSuccess) e = cudaFuncSetAttribute(paged_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  const Scratch s = scratch_at(workspace, sms, BM, p.d);
  paged_tc_kernel<<<sms, NT, kSmem, stream>>>(m.q, m.k, m.v, m.mk, m.mv, p, s, tile_tokens_of(p));
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join(p, 1, s, sms, BM, tile_tokens_of(p), stream);
}

// Whether there are tensor maps: pages of at least 8 tokens (a box starts at a multiple of 8 rows of the swizzled tile), and
// strides that a map takes (below 2^40 bytes; those of 16 bytes and more are multiples of 16 already).
bool tc_supported(const PagedParams& p) {
  const int64_t steps[] = {p.k_page, p.v_page, p.k_token, p.v_token, p.k_head, p.v_head};
  const int sizes[] = {p.n_pages, 1 << p.page_shift, p.h_kv};
  for (int i = 0; i < 6; ++i)
    if ((steps[i] == 0 && sizes[i / 2] > 1) || steps[i] >= (int64_t)1 << 39) return false;
  return p.page_shift >= 3 && p.n_pages >= 1 && p.q_stride < (int64_t)1 << 39;
}

}  // namespace paged
}  // namespace gdn
