// Linear attention with a decay for each head over packed prompts, bf16 inputs, on the tensor cores
// (tcgen05 + TMEM + TMA).
//
// Method: as in linear_simt.cu, with chunks of C = 128 tokens.  With the entering state S (d_v x d_k),
// pw(n) = lambda^n and rho_t = pw(t + 1):
//   O_t = scale rho_t (S q_t + sum_{s <= t} P_ts v_s),   P_ts = pw(t - s) / rho_t  q_t.k_s
//   S  <- pw(n) S + sum_s pw(n - 1 - s) v_s k_s^T
// The scores are divided by rho_t so that both parts of O_t share one accumulator.  rho_t is not let
// below 2^-60 (the quotient must not overflow): a head that decays that far inside a chunk then keeps
// 2^-60 of its entering state where it should keep less, 1e-18 of its size.
//
// A work item is one (segment of a sequence, v-head): its chunks in order.  Products per chunk, all
// M = N = 128 (N = 64 for head sizes up to 64), fp32 accumulators in TMEM:
//   QK   Q K^T             A = Q, B = K (both K-major)                  8 MMAs
//   QS   Q S^T             A = Q, B = S rounded to bf16 (K-major)       8
//   PV   P V               A = P rounded to bf16 (TMEM), B = V          8
//   KV   (W V)^T K         A = the decay-weighted values, transposed, as four bf16 terms (below),
//                          in TMEM, B = K                                 32
// O's operands S and P are rounded once each, as the output itself is; the state is carried in fp32
// registers and never read back from its rounded copy.
//
// The weighted values.  A state at fp32 accuracy needs the weight's 24 bits.  With the weight as three
// bf16 terms w = a + b + c (8 bits each) the product with a bf16 value v splits without error:
//   v a = h + r,  h = bf16(v a), r = v a - h;   v b = m + r',  m = bf16(v b);   l = bf16(v c + r')
// so w v = h + r + m + l up to 2^-25, in five packed bf16 instructions for two values.  (The fp32
// product split into three terms needs a quarter fewer MMAs and three times the instructions: 32,768
// tokens, 32 heads, state only, 135 us against 118; three terms by exact bf16 sums: 178.)
//
// Warpgroups (four warps; registers moved between them by setmaxnreg):
//   0, 1  scores to P, outputs: a thread owns a row t, group 0 the column blocks 0 and 2 of the scores
//         and the first half of the outputs, group 1 the others.  (State only: 0-3 as 2, 3.)
//   2, 3  values to A operands, quarters of 32 tokens in turn: weight, transpose (ldmatrix), split
//   4, 5  the state: a thread owns half a row of S
//   6     one warp issues QK, QS, PV, one KV, one loads the tiles ahead and stores the outputs from the
//         stage of V that they replace, one fetches the work
// Every hand-off is an mbarrier; every wait is bounded.
//
// One CTA per SM stays and takes item after item (clusterlaunchcontrol): the loads, products and tables
// of the next item start while the last chunks of the one before are finished.
//
// Infinite and NaN values.  P V multiplies a later token's value by a score of zero, which gives NaN where
// the recurrence has nothing.  Such a value leaves its row of the state NaN for good, so the state's warps
// see it at an item's end; the outputs it must not reach, at most 127 of a column, are computed again by
// the recurrence behind the block's last item (amend_outputs).  Calls without such values pay one test per
// item (64 prompts of 1556 tokens: 623 to 625 us).  Taking the values out of V's tile ahead of P V was
// slower: seen by the splitting warps 690, by PV's own warp 695, by the work's warp 678; items done a
// second time with V cleaned, 663.
//
// Bound: no single unit.  Per chunk with outputs (about 6,400 clocks) the shared-memory port is busy
// for 4,000 (56 MMAs' operands, the copies, the staging), the tensor pipe for 56 MMAs, and each group's
// loop is about as long as the chunk; at 64 prompts of 1556 tokens, 16/32 heads, the board's power limit
// also holds the clock near 1.8 of 2.07 GHz.  Measured there: 605 us, 4.0 TB/s of 2.45 GB (665 us and
// 4.1 TB/s with entering states; up to 717 us on boards that are held lower); one prompt of 3,277 tokens
// 55 us, of 32,768 state only 115 us (an SM has work for 75% of that, its tensor pipe for 65% of its work).  Measured and left at that first shape: QS issued by the KV warp
// (640 to 690 us) or by the work's warp (683), PV before QS (787), outputs stored from registers (700),
// outputs staged in Q's tile (647), other register shares (609 to 689).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "linear_work.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace {

using namespace tc;
using tcp::kbf16;
using tcp::kWaitNs;

constexpr int C = 128;           // tokens per chunk
constexpr int NWARP = 28, NT = 32 * NWARP;
constexpr int kRegsLaunch = 72;  // a thread's registers at launch, and (below) in its warpgroup's role
constexpr int kRegsRows = 72, kRegsSplit = 56, kRegsState = 96, kRegsControl = 56;
static_assert(2 * kRegsRows + 2 * kRegsSplit + 2 * kRegsState + kRegsControl <= 7 * kRegsLaunch &&
              4 * kRegsSplit + 2 * kRegsState + kRegsControl <= 7 * kRegsLaunch, "what a launch holds");
constexpr uint32_t kTile = 32768, kAtom = 16384;  // 128 rows x 128 bf16: two swizzled atoms of 64 columns

// A work item as the scheduling warp hands it out, in one of two slots with its head's tables.
struct Item {
  int n_chunks;  // -1: no more work
  int t_begin, n_last, h;
  float g;
  int dst, to_local;  // where the state behind the item goes: index of a state in S_out or in `local`; -1: nowhere
  int block;
  const float* S_in;  // entering state, or null (zero)
};

// 32 rows of half a state that an item left all NaN, and the item (its block index).
struct NanRows {
  int block, warp;  // of the state's warps
  uint32_t rows;
};
// An item has at most 8 entries, and three more may be under way when the last steal is decided.
constexpr int kNanMost = 32, kNanSteal = kNanMost - 3 * 8;

// Shared memory: with outputs two stages of [Q | K | V] and the bf16 state (K-major); state only three
// stages of [K | V].  The state's tile (there: a spare one) also stages entering and final states.
// Everything up to CF needs 1024-byte alignment, which the start of dynamic shared memory has here.
template <bool OUT>
struct Lay {
  static constexpr int kStages = OUT ? 2 : 3;
  static constexpr uint32_t Q = 0, K = OUT ? 2 * kTile : 0, V = K + kStages * kTile;
  static constexpr uint32_t S = V + kStages * kTile;
  static constexpr uint32_t CF = S + kTile;      // per slot: pw(31 - j), 32 floats
  static constexpr uint32_t W = CF + 2 * 128;    // per slot: weight terms, 192 words
  static constexpr uint32_t ITEM = W + 2 * 768;  // per slot: the item
  static constexpr uint32_t BARS = ITEM + 2 * 64;
  static constexpr uint32_t STEAL = BARS + 8 * 48;
  static constexpr uint32_t SCRATCH = STEAL + 16;
  static constexpr uint32_t NANS = SCRATCH + 4 * 16;
  static constexpr uint32_t TOTAL = NANS + (OUT ? kNanMost * sizeof(NanRows) : 0);
  static_assert(sizeof(Item) <= 64 && TOTAL <= 232448, "shared memory");
};
// TMEM columns.  With outputs: QK (then P), O, KV, two A buffers; state only: two KV, four A buffers
// ([h | r | m | l] of 32 tokens, 16 columns each).
template <bool OUT>
struct Tmem {
  static constexpr uint32_t cP = 0, cO = 128, cKV = OUT ? 256 : 0, cA = OUT ? 384 : 256;
  static constexpr int kABufs = OUT ? 2 : 4, kKVBufs = OUT ? 1 : 2;
  static constexpr uint32_t ASTEP = 64;
  static_assert(cA + kABufs * ASTEP <= 512, "TMEM");
};

enum Bar { kFull = 0, kEmpty = 3, kAFull = 6, kAFree = 10, kKV = 14, kKVFree = 16, kQK = 18, kP, kOFull, kOFree,
           kSFull, kSFree, kVRead, kStaged = kVRead + 2, kFix = kStaged + 2, kDrainA = kFix + 2, kDrainB, kCorner, kSteal, kItem, kItemFree = kItem + 2,
           kPair = kItemFree + 2 /* one per quad */, kBars = kPair + 4 };
static_assert(kBars <= 48, "barrier area");

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two fp32 operations in one instruction (values as register pairs, the first in the low half).
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Work stealing: asks for a block of this grid that has not been launched yet; its index, if there is
// one, arrives in the 16 bytes at `resp`.
__device__ __forceinline__ void steal_block(void* resp, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(resp)),
               "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ bool stolen_block(const void* resp, int& block) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(resp))
      : "memory");
  block = (int)x;
  return got != 0;
}
// Four 8x8 bf16 tiles, transposed: register i of a thread holds two consecutive rows of tile i's
// column lane / 4.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
// 16 TMEM lanes x 16 columns: registers 2 i and 2 i + 1 are rows lane / 4 and lane / 4 + 8 of column
// 4 i + lane % 4.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Packed bf16 arithmetic, every result rounded once.
constexpr uint32_t kNeg = 0x80008000u;  // flips both signs
__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Whether a bf16 value is infinite or NaN.
__device__ __forceinline__ bool not_finite(uint16_t x) { return (x & 0x7f80u) == 0x7f80u; }
// 32 lanes x 16 columns (thread i -> lane i).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// The weights lambda^back and lambda^(back - 1) of two consecutive tokens (0 at a negative exponent) as
// three packed bf16 terms each, which sum to them exactly.
__device__ __forceinline__ void weight_terms(int back, float g, uint32_t& a, uint32_t& b, uint32_t& c) {
  uint32_t t[2][3];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int e = back - x;
    float w = e < 0 ? 0.f : e == 0 ? 1.f : expf((float)e * g);
#pragma unroll
    for (int y = 0; y < 3; ++y) {
      t[x][y] = __float_as_uint(w) & 0xffff0000u;
      w -= __uint_as_float(t[x][y]);
    }
  }
  a = t[0][0] >> 16 | t[1][0];
  b = t[0][1] >> 16 | t[1][1];
  c = t[0][2] >> 16 | t[1][2];
}
// Registers per thread of the calling warpgroup.
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// What this thread's bulk copies wrote is there.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ Segment segment_of(const LinearWork& p, int block) {
  return p.list ? p.list[block / p.h_v] : only_segment(p, block / p.h_v);
}

// Behind the last item of a block, one warp a row d of a state that is NaN throughout.  In P V an infinite
// or NaN value v_s[d] makes column d NaN for its whole chunk: the zero score of an earlier token times it
// is NaN too.  The outputs of these earlier tokens are computed again by the recurrence; those of the
// chunks before are right, and from s on they are not finite by definition.
__device__ __forceinline__ void amend_outputs(const LinearWork& p, const NanRows& nan, int row) {
  if (nan.warp >= 4 || !(nan.rows >> row & 1)) return;  // (both halves of a row are NaN then)
  const Segment s = segment_of(p, nan.block);
  const int h = nan.block % p.h_v, d = 32 * nan.warp + row, lane = threadIdx.x & 31;
  const size_t v_step = (size_t)p.h_v * p.d_v, k_step = (size_t)p.h_k * p.d_k;
  const size_t v_at = (size_t)s.t_begin * v_step + (size_t)h * p.d_v + d;
  const size_t k_at = (size_t)s.t_begin * k_step + (size_t)(h / (p.h_v / p.h_k)) * p.d_k + 4 * lane;
  const uint16_t* v = static_cast<const uint16_t*>(p.v) + v_at;
  const ItemState state = item_state(p, s, h, true);
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (state.S_in && 4 * lane < p.d_k) S = *reinterpret_cast<const float4*>(state.S_in + (size_t)d * p.d_k + 4 * lane);
  // (no output of a row that enters with infinities or NaN is finite)
  if (__any_sync(0xffffffffu, !isfinite(S.x) || !isfinite(S.y) || !isfinite(S.z) || !isfinite(S.w))) return;
  int first = s.len;  // the first such token
#pragma unroll 1
  for (int t0 = 0; t0 < s.len && first == s.len; t0 += 32) {
    const unsigned found = __ballot_sync(0xffffffffu, t0 + lane < s.len && not_finite(v[(t0 + lane) * v_step]));
    if (found) first = t0 + __ffs(found) - 1;
  }
  const int begin = first / C * C;
  if (first == s.len || first == begin) return;
  auto four = [&](const void* x, int t) {
    uint2 u = make_uint2(0u, 0u);
    if (4 * lane < p.d_k) u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x) + k_at + t * k_step);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
  };
  const DecayStep f = decay_step(p.log_decay[h], 1);
  auto step = [&](int t) {
    const float x = __uint_as_float((uint32_t)v[t * v_step] << 16);
    const float4 k = four(p.k, t);
    S = make_float4(f(S.x, x * k.x), f(S.y, x * k.y), f(S.z, x * k.z), f(S.w, x * k.w));
  };
#pragma unroll 4
  for (int t = 0; t < begin; ++t) step(t);
#pragma unroll 1
  for (int t = begin; t < first; ++t) {
    step(t);
    const float4 q = four(p.q, t);
    float o = fmaf(S.x, q.x, fmaf(S.y, q.y, fmaf(S.z, q.z, S.w * q.w)));
#pragma unroll
    for (int i = 16; i; i >>= 1) o += __shfl_xor_sync(0xffffffffu, o, i);
    if (lane == 0) static_cast<__nv_bfloat16*>(p.O)[v_at + t * v_step] = __float2bfloat16_rn(p.scale * o);
  }
}
// The half row of the final state, all NaN, in the place of the entering one.
__device__ __forceinline__ void nan_row(const LinearWork& p, const NanRows& nan, int row) {
  if (!(nan.rows >> row & 1)) return;
  const ItemState state = item_state(p, segment_of(p, nan.block), nan.block % p.h_v, true);
  if (state.dst < 0) return;
  float* S = (state.to_local ? p.local : p.S_out) + ((size_t)state.dst * p.d_v + 32 * (nan.warp & 3) + row) * p.d_k;
  const int lane = threadIdx.x & 31;
  for (int c = 64 * (nan.warp >> 2) + lane; c < min(p.d_k, 64 * (nan.warp >> 2) + 64); c += 32) S[c] = __int_as_float(0x7fffffff);
}

// OUT: outputs and the final state; otherwise the states of the items alone (to S_out when a sequence
// is one segment, to `local`, from zero, when it is cut).
template <bool OUT>
__global__ void __launch_bounds__(NT, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                     const __grid_constant__ CUtensorMap map_s, const __grid_constant__ CUtensorMap map_local,
                     const LinearWork p) {
  using L = Lay<OUT>;
  using TM = Tmem<OUT>;
  constexpr int kStages = L::kStages;
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BARS);
  int* scratch = reinterpret_cast<int*>(sm + L::SCRATCH);
  volatile int* dead = scratch;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scratch + 1);
  int* issued = scratch + 2;  // chunks whose loads were issued
  int* n_nans = scratch + 3;
  NanRows* nans = reinterpret_cast<NanRows*>(sm + L::NANS);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = warp >> 2, quad = warp & 3;
  const int dkp = p.d_k <= 64 ? 64 : 128, dvp = p.d_v <= 64 ? 64 : 128;  // columns that the products cover

  if (smem_u32(sm) & 1023u) {  // (the swizzled tiles could not be addressed)
    if (tid == 0) atomicExch(p.status, GDN_ERR_CUDA);
    return;
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int b = 0; b < kBars; ++b) {
      int count = 1;
      if (b >= kEmpty && b < kEmpty + 3) count = OUT ? 2 : 1;  // the issuing warps' commits
      if (b >= kAFull && b < kAFull + 4) count = 4;            // the warps of a splitting group
      if (b == kP || b == kOFree || b == kSFull || b == kKVFree || b == kKVFree + 1 ||
          (b >= kVRead && b < kFix + 2) || b == kCorner)
        count = 8;
      if (b >= kItemFree && b < kItemFree + 2) count = OUT ? 27 : 26;  // every warp that reads items
      if (b >= kPair) count = 2;
      mbar_init(&bar[b], count);
    }
    mbar_fence_init();
    *dead = 0;
    *issued = 0;
    *n_nans = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
  auto wait = [&](int b, int parity, uint64_t limit = kWaitNs) {
    if (mbar_wait(&bar[b], (uint32_t)(parity & 1), limit)) return true;
    *dead = 1;
    return false;
  };
  auto arrive = [&](int b) {  // one arrival per warp, behind what its threads did before
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[b]);
  };
  auto item_at = [&](int k) { return reinterpret_cast<const Item*>(sm + L::ITEM + 64 * (k & 1)); };
  // Item k is there (n_chunks < 0: the work is done).  (A whole item may pass meanwhile.)
  constexpr uint64_t kItemNs = 8 * kWaitNs;
  auto get_item = [&](int k) { return wait(kItem + (k & 1), k >> 1, kItemNs) && item_at(k)->n_chunks >= 0; };
  auto release_item = [&](int k) { arrive(kItemFree + (k & 1)); };
  // Every role counts the chunks of all its items, gc: stages, accumulators and phases go by that.  A
  // barrier's next phase but one never completes before every waiter has seen this one: its arrivals
  // follow, through other barriers, from what the waiter does next.  (Two each, by turns: kVRead, since
  // the splitting warps can be done with two chunks' values before the rows' warps look; kStaged, two
  // chunks' outputs before the loading warp does; kFix, the ends of two one-chunk items before the warp
  // that issues PV does.)

  if (OUT && group < 2) {
    // ------------------------------------------------------------ scores to P, outputs
    const int t = 32 * quad + lane;
    bool ok = true;
    for (int k = 0, gc = 0; ok && get_item(k); ++k) {
      const Item& it = *item_at(k);
      const float* cf = reinterpret_cast<const float*>(sm + L::CF + 128 * (k & 1));
      const int n_chunks = it.n_chunks, n_last = it.n_last, h = it.h, t_begin = it.t_begin;
      const float g = it.g;
      const float rho = fmaxf(expf((float)(t + 1) * g), 8.673617379884035e-19f);  // 2^-60
      const float inv = 1.f / rho, f = rho * p.scale;
      // The factor of a score is lambda^(t - s) / rho_t = rf cf[j] for column j of a block: rf =
      // lambda^(t - 32 b - 31) / rho_t, and cf[j] = lambda^(31 - j).  On the diagonal (t - 32 b = lane)
      // rf's power has a negative exponent; where rf could leave the fp32 range (a decay below e^-1.4
      // per token) the block takes cf[31 - lane + j] instead.
      const bool steep = !(cf[0] > 1e-19f);
      // Where no rho_t of the chunk is held back, the factor is lambda^-(s + 1), the column's alone.
      const bool gentle = expf((float)C * g) >= 8.673617379884035e-19f;
      float rc[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) rc[i] = gentle ? expf(-(float)(32 * (2 * i + group) + 32) * g) : 0.f;
      float rf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int b = 2 * i + group;
        rf[i] = b < quad ? expf((float)(t - 32 * b - 31) * g) * inv : steep ? inv : inv / cf[lane];
      }
      for (int c = 0; c < n_chunks; ++c, ++gc) {
        const int n = c + 1 < n_chunks ? C : n_last;
        if (!(ok = wait(kQK, gc))) break;
        tc_fence_after();
        // Blocks of 32 columns: the row's blocks before `quad` whole, its own up to the diagonal, none
        // behind.  P overwrites scores that the other warp of this quad may still be reading, so both
        // read and round first.
        uint32_t o[2][16];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int b = 2 * i + group;
          if (b <= quad) {
            float x[32];
            tmem_ld32(tmem + lane_base + TM::cP + 32 * b, x);
            tmem_ld_wait();
            if (gentle) {
              const uint64_t rf2 = pair(rc[i], rc[i]);
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(cf + j);
                float y0, y1, y2, y3;
                unpair(mul2(pair(x[j], x[j + 1]), mul2(rf2, w.x)), y0, y1);
                unpair(mul2(pair(x[j + 2], x[j + 3]), mul2(rf2, w.y)), y2, y3);
                o[i][j / 2] = pack_bf16(y0, y1);
                o[i][j / 2 + 1] = pack_bf16(y2, y3);
              }
              if (b == quad) {
#pragma unroll
                for (int j = 0; j < 32; j += 2) o[i][j / 2] &= lane > j ? 0xffffffffu : lane == j ? 0xffffu : 0u;
              }
            } else if (b < quad || !steep) {
              const uint64_t rf2 = pair(rf[i], rf[i]);
              const int seen = b < quad ? 31 : lane;  // the last column that counts
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(cf + j);
                float y0, y1, y2, y3;
                unpair(mul2(pair(x[j], x[j + 1]), mul2(rf2, w.x)), y0, y1);
                unpair(mul2(pair(x[j + 2], x[j + 3]), mul2(rf2, w.y)), y2, y3);
                o[i][j / 2] = pack_bf16(j <= seen ? y0 : 0.f, j + 1 <= seen ? y1 : 0.f);
                o[i][j / 2 + 1] = pack_bf16(j + 2 <= seen ? y2 : 0.f, j + 3 <= seen ? y3 : 0.f);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const float y0 = j <= lane ? x[j] * (cf[31 - lane + j] * rf[i]) : 0.f;
                const float y1 = j + 1 <= lane ? x[j + 1] * (cf[32 - lane + j] * rf[i]) : 0.f;
                o[i][j / 2] = pack_bf16(y0, y1);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[i][j] = 0u;
          }
        }
        arrive(kPair + quad);
        if (!(ok = wait(kPair + quad, gc))) break;
        tmem_st16(tmem + lane_base + TM::cP + 16 * group, o[0]);
        tmem_st16(tmem + lane_base + TM::cP + 32 + 16 * group, o[1]);
        tmem_st_wait();
        tc_fence_before();
        arrive(kP);
        if (!(ok = wait(kOFull, gc))) break;
        tc_fence_after();
        // The outputs, rounded, into the stage of V, once the splitting warps have read it too
        if (!(ok = wait(kVRead + (gc & 1), gc >> 1))) break;
        unsigned char* stage = sm + L::V + (gc & 1) * kTile;
        if (64 * group < dvp) {
          const uint64_t f2 = pair(f, f);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float x[32];
            tmem_ld32(tmem + lane_base + TM::cO + 64 * group + 32 * b, x);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float y0, y1;
                unpair(mul2(f2, pair(x[j + 2 * e], x[j + 2 * e + 1])), y0, y1);
                y[e] = pack_bf16(y0, y1);
              }
              *reinterpret_cast<uint4*>(stage + kbf16(t, 64 * group + 32 * b + j, 128)) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
        }
        tc_fence_before();
        arrive(kOFree);
        // (of a part of a chunk the rows behind its end are not this sequence's: row by row)
        if (n < C && 8 * (lane & 7) + 64 * group < p.d_v) {
          const int col = 64 * group + 8 * (lane & 7);
          for (int row = 32 * quad + (lane >> 3); row < min(n, 32 * quad + 32); row += 4)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.O) + ((size_t)(t_begin + c * C + row) * p.h_v + h) * p.d_v + col) =
                *reinterpret_cast<const uint4*>(stage + kbf16(row, col, 128));
        }
        fence_async_smem();
        arrive(kStaged + (gc & 1));
      }
      release_item(k);
    }
  } else if (group < 4) {
    // ------------------------------------------------------------ values to A operands
    regs_dec<kRegsSplit>();
    constexpr int kPer = 4 / TM::kABufs;  // quarters of a chunk per group
    const int buf = OUT ? group - 2 : group;
    const bool rows = 32 * quad < dvp;
    // this lane's part of the ldmatrix addresses: tile lane / 8 of (8 d) x (8 tokens), token lane % 8
    const int lm_tok = (lane & 7) + 8 * (lane >> 4), lm_d = 32 * quad + 8 * ((lane >> 3) & 1);
    const uint32_t at = tmem + lane_base + TM::cA + buf * TM::ASTEP;
    bool ok = true;
    for (int k = 0, gc = 0; ok && get_item(k); ++k) {
      const int n_chunks = item_at(k)->n_chunks, n_last = item_at(k)->n_last;
      const uint32_t* table = reinterpret_cast<const uint32_t*>(sm + L::W + 768 * (k & 1)) + 12 * (lane & 3);
      for (int c = 0; c < n_chunks && ok; ++c, ++gc) {
        const int st = gc % kStages, n = c + 1 < n_chunks ? C : n_last;
        if (!(ok = wait(kFull + st, gc / kStages))) break;
#pragma unroll 1
        for (int i = 0; i < kPer; ++i) {
          const int q = buf + TM::kABufs * i, m = gc * kPer + i;
          uint32_t x[4][4];  // tiles of 16 rows x 16 tokens: (rows +0, tokens +0), (+0, +16), (+16, +0), (+16, +16)
          uint32_t wt[3][4];
          if (rows) {
            const uint32_t vt = smem_u32(sm + L::V + st * kTile) + (uint32_t)(32 * q + lm_tok) * 128u;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int d = lm_d + 16 * (b >> 1);
              ldmatrix_x4_trans(vt + (d >> 6) * kAtom + 2048 * (b & 1) + ((((d & 63) >> 3) ^ (lm_tok & 7)) << 4), x[b]);
            }
            if (n == C) {
#pragma unroll
              for (int y = 0; y < 3; ++y) {
                const uint4 u = *reinterpret_cast<const uint4*>(table + 48 * q + 4 * y);
                wt[y][0] = u.x; wt[y][1] = u.y; wt[y][2] = u.z; wt[y][3] = u.w;
              }
            } else {  // the weights count back from the last token; a row behind it may hold anything
              const float g = item_at(k)->g;
#pragma unroll
              for (int e = 0; e < 4; ++e) weight_terms(n - 1 - (32 * q + 8 * e + 2 * (lane & 3)), g, wt[0][e], wt[1][e], wt[2][e]);
#pragma unroll
              for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int tok = 32 * q + 16 * (b & 1) + 8 * (j >> 1) + 2 * (lane & 3);
                  x[b][j] = tok >= n ? 0u : tok + 1 >= n ? x[b][j] & 0xffffu : x[b][j];
                }
            }
          }
          if (OUT && i + 1 == kPer) arrive(kVRead + (gc & 1));
          if (m > 0 && !(ok = wait(kAFree + buf, m - 1))) break;
          tc_fence_after();
          if (rows) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t t[4][8];  // h, r, m, l of 16 rows x 32 tokens
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint32_t v = x[2 * half + (j >> 2)][j & 3], *w = &wt[0][j >> 1];
                t[0][j] = bmul2(v, w[0]);
                t[1][j] = bfma2(v, w[0], t[0][j] ^ kNeg);
                t[2][j] = bmul2(v, w[4]);
                t[3][j] = bfma2(v, w[8], bfma2(v, w[4], t[2][j] ^ kNeg));
              }
#pragma unroll
              for (int y = 0; y < 4; ++y) tmem_st_16x128b_x4(at + ((uint32_t)(16 * half) << 16) + 16 * y, t[y]);
            }
            tmem_st_wait();
          }
          tc_fence_before();
          arrive(kAFull + buf);
        }
      }
      release_item(k);
    }
  } else if (group < 6) {
    // ------------------------------------------------------------ the state
    regs_inc<kRegsState>();
    const int hw = group - 4;
    const int r = 32 * quad + lane;  // row of S
    const bool mine = 32 * quad < dvp && 64 * hw < dkp;
    // Entering and final states pass through a corner of the state's tile, 32 rows x 32 columns per warp
    // (16-byte chunks swizzled by row, as a tensor copy with 128-byte swizzle has them), so that global
    // memory sees whole 128-byte lines.
    float* corner = reinterpret_cast<float*>(sm + L::S) + 1024 * (warp - 16);
    const int my_chunk = lane & 7, my_row = lane >> 3;
    float s[64];
    auto publish_state = [&]() {  // the state, rounded to bf16, as QS's B operand
      if (mine) {
#pragma unroll
        for (int j = 0; j < 64; j += 8)
          *reinterpret_cast<uint4*>(sm + L::S + kbf16(r, 64 * hw + j, 128)) =
              make_uint4(pack_bf16(s[j], s[j + 1]), pack_bf16(s[j + 2], s[j + 3]), pack_bf16(s[j + 4], s[j + 5]),
                         pack_bf16(s[j + 6], s[j + 7]));
      }
      fence_async_smem();
      arrive(kSFull);
    };
    bool ok = true;
    for (int k = 0, gc = 0, fixes = 0; ok && get_item(k); ++k) {
      const int n_chunks = item_at(k)->n_chunks, n_last = item_at(k)->n_last;
      if (const float* S_in = item_at(k)->S_in) {
        if (OUT && p.early) grid_dep_wait();  // the entering states
        // (all loads under way at once: s holds them in the order of memory first)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int row = 4 * (i & 7) + my_row, col = 64 * hw + 32 * (i >> 3) + 4 * my_chunk;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (32 * quad + row < p.d_v && col < p.d_k)
            x = *reinterpret_cast<const float4*>(S_in + (size_t)(32 * quad + row) * p.d_k + col);
          s[4 * i] = x.x; s[4 * i + 1] = x.y; s[4 * i + 2] = x.z; s[4 * i + 3] = x.w;
        }
        bulk_wait_read_all();  // (the final state before this one has left the corner)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + my_row;
            *reinterpret_cast<float4*>(corner + 32 * row + 4 * (my_chunk ^ (row & 7))) =
                make_float4(s[32 * j + 4 * i], s[32 * j + 4 * i + 1], s[32 * j + 4 * i + 2], s[32 * j + 4 * i + 3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(corner + 32 * lane + 4 * (i ^ (lane & 7)));
            s[32 * j + 4 * i] = x.x; s[32 * j + 4 * i + 1] = x.y; s[32 * j + 4 * i + 2] = x.z; s[32 * j + 4 * i + 3] = x.w;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 64; ++j) s[j] = 0.f;
        bulk_wait_read_all();
      }
      if (OUT) {  // (the rounded state is written over other warps' corners)
        arrive(kCorner);
        if (!(ok = wait(kCorner, k))) break;
        if (n_chunks > 0) publish_state();
      }
      for (int c = 0; c < n_chunks; ++c, ++gc) {
        const int st = gc % kStages, kv = gc % TM::kKVBufs, n = c + 1 < n_chunks ? C : n_last;
        if (n < C) {
          // rows behind the last token: another sequence's, or none; they may hold anything
          if (!(ok = wait(kFull + st, gc / kStages))) break;
          const int per_row = (dkp + dvp) / 8;
          for (int e = tid - 512; e < (C - n) * per_row; e += 256) {
            const int row = n + e / per_row, x = e % per_row;
            unsigned char* tile = x < dkp / 8 ? sm + L::K + st * kTile : sm + L::V + st * kTile;
            const int col = x < dkp / 8 ? x : x - dkp / 8;
            *reinterpret_cast<uint4*>(tile + (col >> 3) * kAtom + row * 128 + (col & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_async_smem();
          arrive(kFix + (fixes & 1));
          ++fixes;
        }
        if (!(ok = wait(kKV + kv, gc / TM::kKVBufs))) break;
        tc_fence_after();
        if (mine) {
          const DecayStep f = decay_step(item_at(k)->g, n);
          const uint32_t at = tmem + lane_base + TM::cKV + 128 * kv + 64 * hw;
          const uint64_t m = f.near1 ? pair(f.f1, f.f1) : pair(f.f, f.f);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            float x[16];
            tmem_ld16(at + 16 * b, x);
            tmem_ld_wait();
            if (f.near1) {
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const uint64_t a = pair(s[16 * b + j], s[16 * b + j + 1]);
                unpair(fma2(a, m, add2(a, pair(x[j], x[j + 1]))), s[16 * b + j], s[16 * b + j + 1]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 16; j += 2)
                unpair(fma2(pair(s[16 * b + j], s[16 * b + j + 1]), m, pair(x[j], x[j + 1])), s[16 * b + j], s[16 * b + j + 1]);
            }
          }
        }
        tc_fence_before();
        arrive(kKVFree + kv);
        if (OUT) {  // (the tile's readers are done: it takes the next rounding, or the final state's corners)
          if (!(ok = wait(kSFree, gc))) break;
          if (c + 1 < n_chunks) publish_state();
        }
      }
      if (!ok) break;
      if (OUT && __any_sync(0xffffffffu, mine && s[0] != s[0])) {
        // Rows that are NaN throughout, as an infinite or NaN value leaves them, are looked at behind the
        // last item (amend_outputs), from their entering state: S_out may be its place, and keeps it till then.
        bool all = mine;
#pragma unroll
        for (int j = 0; j < 64; ++j) all = all && (64 * hw + j >= p.d_k || s[j] != s[j]);
        const unsigned rows = __ballot_sync(0xffffffffu, all && r < p.d_v);
        if (lane == 0 && rows) nans[atomicAdd(n_nans, 1)] = NanRows{item_at(k)->block, warp - 16, rows};
        if (const float* S_in = item_at(k)->S_in) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if ((rows >> lane & 1) && 64 * hw + j < p.d_k) s[j] = S_in[(size_t)r * p.d_k + 64 * hw + j];
        }
      }
      if (item_at(k)->dst >= 0 && mine) {
        const CUtensorMap* map = item_at(k)->to_local ? &map_local : &map_s;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (j) bulk_wait_read_all();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(corner + 32 * lane + 4 * (i ^ (lane & 7))) =
                make_float4(s[32 * j + 4 * i], s[32 * j + 4 * i + 1], s[32 * j + 4 * i + 2], s[32 * j + 4 * i + 3]);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(map, corner, 64 * hw + 32 * j, 32 * quad, item_at(k)->dst);
            bulk_commit();
          }
        }
      }
      release_item(k);
    }
    bulk_wait_read_all();
  } else {
    regs_dec<kRegsControl>();
    if (quad == 0) {
      // ---------------------------------------------------------- QK, QS, PV
      if constexpr (OUT) {
        const uint32_t idQK = idesc_bf16(128, 128, false, false), idQS = idesc_bf16(128, dvp, false, false),
                       idPV = idesc_bf16(128, dvp, false, true);
        const int nk = (p.d_k + 15) / 16;
        const uint64_t dQ0 = sdesc_sw128(smem_u32(sm + L::Q), 16, 1024), dK0 = sdesc_sw128(smem_u32(sm + L::K), 16, 1024),
                       dS = sdesc_sw128(smem_u32(sm + L::S), 16, 1024), dV0 = sdesc_sw128(smem_u32(sm + L::V), kAtom, 1024);
        int k = -1, left = 0, fixes = 0;  // item, its chunks not yet begun
        bool ok = true;
        // The next chunk's item, past items of no tokens; false when the work is done.
        auto next_chunk = [&]() {
          while (left == 0) {
            if (k >= 0) release_item(k);
            if (!get_item(++k)) return false;
            left = item_at(k)->n_chunks;
          }
          --left;
          return true;
        };
        auto issue_qk = [&](int gc) {
          if (!wait(kFull + (gc & 1), gc >> 1)) return false;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t st = (uint64_t)((gc & 1) * kTile) >> 4;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < nk) {
                const uint64_t off = st + (uint64_t)(((i >> 2) * kAtom + (i & 3) * 32) >> 4);
                mma_bf16(tmem + TM::cP, dQ0 + off, dK0 + off, idQK, i > 0);
              }
            mma_commit(&bar[kQK]);
          }
          __syncwarp();
          return true;
        };
        if (next_chunk() && issue_qk(0)) {
          for (int gc = 0; ok; ++gc) {
            const uint64_t st = (uint64_t)((gc & 1) * kTile) >> 4;
            const bool part = left == 0 && item_at(k)->n_last < C;
            if (!wait(kSFull, gc)) break;
            if (gc > 0 && !wait(kOFree, gc - 1)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < nk) {
                  const uint64_t off = (uint64_t)(((i >> 2) * kAtom + (i & 3) * 32) >> 4);
                  mma_bf16(tmem + TM::cO, dQ0 + st + off, dS + off, idQS, i > 0);
                }
              mma_commit(&bar[kSFree]);
            }
            __syncwarp();
            if (!wait(kP, gc)) break;
            if (part) {
              if (!wait(kFix + (fixes & 1), fixes >> 1)) break;
              ++fixes;
            }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                mma_bf16_ts(tmem + TM::cO, tmem + TM::cP + 8 * i, dV0 + st + (uint64_t)((i * 2048) >> 4), idPV, 1);
              mma_commit(&bar[kOFull]);
              mma_commit(&bar[kEmpty + (gc & 1)]);
            }
            __syncwarp();
            ok = next_chunk() && issue_qk(gc + 1);
          }
        }
        if (elect_one()) mma_commit(&bar[kDrainA]);
        __syncwarp();
        mbar_wait(&bar[kDrainA], 0, kWaitNs);
      }
    } else if (quad == 1) {
      // ---------------------------------------------------------- KV
      const uint32_t idKV = idesc_bf16(128, dkp, false, true);
      bool ok = true;
      for (int k = 0, gc = 0, fixes = 0; ok && get_item(k); ++k) {
        const int n_chunks = item_at(k)->n_chunks;
        for (int c = 0; c < n_chunks && ok; ++c, ++gc) {
          const int st = gc % kStages, kv = gc % TM::kKVBufs;
          const uint32_t d = tmem + TM::cKV + 128 * kv;
          if (!(ok = wait(kFull + st, gc / kStages))) break;
          if (c + 1 == n_chunks && item_at(k)->n_last < C) {
            if (!(ok = wait(kFix + (fixes & 1), fixes >> 1))) break;
            ++fixes;
          }
          if (gc >= TM::kKVBufs && !(ok = wait(kKVFree + kv, gc / TM::kKVBufs - 1))) break;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            const int buf = q % TM::kABufs, m = gc * (4 / TM::kABufs) + q / TM::kABufs;
            if (!(ok = wait(kAFull + buf, m))) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t dK = sdesc_sw128(smem_u32(sm + L::K + st * kTile), kAtom, 1024);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint64_t b = dK + (uint64_t)(((32 * q + 16 * i) * 128) >> 4);
                const uint32_t a = tmem + TM::cA + buf * TM::ASTEP + 8 * i;
                mma_bf16_ts(d, a + 48, b, idKV, q > 0 || i > 0);
                mma_bf16_ts(d, a + 32, b, idKV, 1);
                mma_bf16_ts(d, a + 16, b, idKV, 1);
                mma_bf16_ts(d, a, b, idKV, 1);
              }
              mma_commit(&bar[kAFree + buf]);
              if (q == 3) {
                mma_commit(&bar[kKV + kv]);
                mma_commit(&bar[kEmpty + st]);
              }
            }
            __syncwarp();
          }
        }
        release_item(k);
      }
      if (elect_one()) mma_commit(&bar[kDrainB]);
      __syncwarp();
      mbar_wait(&bar[kDrainB], 0, kWaitNs);
    } else if (quad == 2) {
      // ---------------------------------------------------------- loads, and stores of whole chunks
      if (lane == 0) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
        if (OUT) {
          tma_prefetch_desc(&map_q);
          tma_prefetch_desc(&map_o);
        }
      }
      const uint32_t bytes = (uint32_t)((OUT ? 2 : 1) * dkp + dvp) * 256u;
      // Outputs staged in the two stages of V: first token and head, or h = -1 (part of a chunk, stored
      // by the warps that staged it).
      int t_old = 0, h_old = -1, t_new = 0, h_new = -1;
      auto store = [&](int gc) {  // chunk gc's outputs, the older of the two, out of their stage, which is then free
        if (!wait(kStaged + (gc & 1), gc >> 1)) return false;
        if (lane == 0 && h_old >= 0) {
          for (int x = 0; x < dvp; x += 64)
            tma_store_3d(&map_o, sm + L::V + (gc & 1) * kTile + (x >> 6) * kAtom, x, h_old, t_old);
          bulk_commit();
          bulk_wait_read_all();
        }
        __syncwarp();
        return true;
      };
      bool ok = true;
      int gc = 0;
      for (int k = 0; ok && get_item(k); ++k) {
        const int n_chunks = item_at(k)->n_chunks, h = item_at(k)->h, hk = h / (p.h_v / p.h_k);
        int t0 = item_at(k)->t_begin;
        const bool part = item_at(k)->n_last < C;
        for (int c = 0; c < n_chunks; ++c, ++gc, t0 += C) {
          const int st = gc % kStages;
          if (gc >= kStages && !(ok = wait(kEmpty + st, gc / kStages - 1))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar[kFull + st], bytes);
            for (int x = 0; x < dkp; x += 64) {
              if (OUT) tma_load_3d(sm + L::Q + st * kTile + (x >> 6) * kAtom, &map_q, &bar[kFull + st], x, hk, t0);
              tma_load_3d(sm + L::K + st * kTile + (x >> 6) * kAtom, &map_k, &bar[kFull + st], x, hk, t0);
            }
          }
          __syncwarp();
          if (OUT) {
            if (gc >= 2) ok = store(gc - 2);
            t_old = t_new;
            h_old = h_new;
            t_new = t0;
            h_new = c + 1 == n_chunks && part ? -1 : h;
          }
          if (lane == 0) {  // (loaded all the same, so that the stage's bytes are whole when a wait gave up)
            for (int x = 0; x < dvp; x += 64)
              tma_load_3d(sm + L::V + st * kTile + (x >> 6) * kAtom, &map_v, &bar[kFull + st], x, h, t0);
          }
          if (lane == 0) *issued = gc + 1;
          __syncwarp();
          if (!ok) break;
        }
        release_item(k);
      }
      if (OUT && !*dead) {
        if (gc >= 2 && store(gc - 2)) {
          t_old = t_new;
          h_old = h_new;
          store(gc - 1);
        } else if (gc == 1) {
          t_old = t_new;
          h_old = h_new;
          store(0);
        }
      }
    } else {
      // ---------------------------------------------------------- the work
      int block = blockIdx.x, k = 0;
      bool ok = true;
      if (p.list) grid_dep_wait();  // the plan
      for (int steals = 0; ok; ++steals) {
        const int h = block % p.h_v, u = block / p.h_v;
        const Segment s = p.list ? p.list[u] : only_segment(p, u);
        if (!p.list && block == 0 && lane == 0 && s.seq < 0) atomicExch(p.status, GDN_ERR_SHAPE);
        if (s.seq >= 0 && !(p.local_only && s.seg + 1 == s.n_seg)) {
          if (k >= 2 && !(ok = wait(kItemFree + (k & 1), (k >> 1) - 1, kItemNs))) break;
          const float g = p.log_decay[h];
          float* cf = reinterpret_cast<float*>(sm + L::CF + 128 * (k & 1));
          cf[lane] = lane == 31 ? 1.f : expf((float)(31 - lane) * g);
          // Weight terms of a whole chunk: word 12 (4 q + j) + 4 term + e holds those of tokens
          // 32 q + 8 e + 2 j + {0, 1}.
          uint32_t* wtab = reinterpret_cast<uint32_t*>(sm + L::W + 768 * (k & 1));
#pragma unroll 1
          for (int i = lane; i < 64; i += 32) {
            const int q = i >> 4, j = (i >> 2) & 3, e = i & 3;
            uint32_t* w = wtab + 12 * (4 * q + j) + e;
            weight_terms(C - 1 - (32 * q + 8 * e + 2 * j), g, w[0], w[4], w[8]);
          }
          if (lane == 0) {
            Item* it = reinterpret_cast<Item*>(sm + L::ITEM + 64 * (k & 1));
            const ItemState state = item_state(p, s, h, OUT);
            it->n_chunks = (s.len + C - 1) / C;
            it->t_begin = s.t_begin;
            it->n_last = s.len > 0 ? (s.len - 1) % C + 1 : C;
            it->h = h;
            it->g = g;
            it->S_in = state.S_in;
            it->to_local = state.to_local;
            it->dst = state.dst;
            it->block = block;
            if (it->S_in) bulk_prefetch_l2(it->S_in, (uint32_t)(p.d_v * p.d_k * 4));
          }
          arrive(kItem + (k & 1));
          ++k;
        }
        // (CTAs that were launched early take nothing from those that start when the kernel ahead ends)
        if (p.early) grid_dep_wait();
        // (with many rows to look at again, this block ends, and others are launched for what is left)
        if (OUT && *static_cast<volatile int*>(n_nans) >= kNanSteal) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar[kSteal], 16);
          steal_block(sm + L::STEAL, &bar[kSteal]);
        }
        if (!(ok = wait(kSteal, steals))) break;
        if (!stolen_block(sm + L::STEAL, block)) break;
        fence_async_smem();  // (the answer's bytes are read before the next one is asked for)
        __syncwarp();
      }
      if (ok && (k < 2 || wait(kItemFree + (k & 1), (k >> 1) - 1, kItemNs))) {
        if (lane == 0) reinterpret_cast<Item*>(sm + L::ITEM + 64 * (k & 1))->n_chunks = -1;
        arrive(kItem + (k & 1));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*dead) {
    // A wait gave up: let the loads in flight land (each wait bounded; the MMAs were drained by their
    // issuing warps), then report.  The results are unspecified.
    if (tid == 0) {
      for (int c = max(0, *issued - kStages); c < *issued; ++c)
        mbar_wait(&bar[kFull + c % kStages], (uint32_t)((c / kStages) & 1), kWaitNs);
      atomicExch(p.status, GDN_ERR_TIMEOUT);
    }
    __syncthreads();
  } else if (OUT && *n_nans > 0) {
    bulk_wait_all();  // what this thread's copies store is there
    __syncthreads();
    if (group == 4 || group == 5)
      for (int i = warp - 16; i < 32 * *n_nans; i += 8) amend_outputs(p, nans[i >> 5], i & 31);
    __syncthreads();
    if (group == 4 || group == 5)
      for (int i = warp - 16; i < 32 * *n_nans; i += 8) nan_row(p, nans[i >> 5], i & 31);
  }
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// [T][heads][d] as a 3-D tensor, boxes of 64 elements x one head x 128 tokens; elements past d and
// tokens past T read as zero.
bool make_map_heads(CUtensorMap* m, const void* base, int tokens, int heads, int d) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
  cuuint32_t box[3] = {64, 1, C};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// fp32 states [count][d_v][d_k], boxes of 32 x 32.
bool make_map_states(CUtensorMap* m, const void* base, size_t count, int d_v, int d_k) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d_k, (cuuint64_t)d_v, (cuuint64_t)count};
  cuuint64_t strides[2] = {(cuuint64_t)d_k * 4, (cuuint64_t)d_v * d_k * 4};
  cuuint32_t box[3] = {32, 32, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernels are launched with the registers that the warpgroups' shares add up to (with fewer, a
// warpgroup that asks for more would wait): checked once.
cudaError_t check_registers() {
  static std::atomic<bool> checked{false};
  if (checked.load(std::memory_order_acquire)) return cudaSuccess;
  const void* kernels[] = {reinterpret_cast<const void*>(linear_tc_kernel<true>),
                           reinterpret_cast<const void*>(linear_tc_kernel<false>)};
  for (const void* kernel : kernels) {
    cudaFuncAttributes have;
    const cudaError_t e = cudaFuncGetAttributes(&have, kernel);
    if (e != cudaSuccess) return e;
    if (have.numRegs != kRegsLaunch) return cudaErrorInvalidKernelImage;
  }
  checked.store(true, std::memory_order_release);
  return cudaSuccess;
}

template <bool OUT>
cudaError_t launch_items(const LinearWork& p, int units, cudaStream_t stream) {
  CUtensorMap mq{}, mk, mv, mo{}, ms, ml{};
  if ((OUT && (!make_map_heads(&mq, p.q, p.total_tokens, p.h_k, p.d_k) ||
               !make_map_heads(&mo, p.O, p.total_tokens, p.h_v, p.d_v))) ||
      !make_map_heads(&mk, p.k, p.total_tokens, p.h_k, p.d_k) ||
      !make_map_heads(&mv, p.v, p.total_tokens, p.h_v, p.d_v) ||
      !make_map_states(&ms, p.S_out, (size_t)p.n_seqs * p.h_v, p.d_v, p.d_k) ||
      (p.cut_units > 0 && !make_map_states(&ml, p.local, (size_t)p.cut_units * p.h_v, p.d_v, p.d_k)))
    return cudaErrorInvalidValue;
  // (in each call: the attribute belongs to the current context)
  const cudaError_t e =
      cudaFuncSetAttribute(linear_tc_kernel<OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<OUT>::TOTAL);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units * p.h_v);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = Lay<OUT>::TOTAL;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, linear_tc_kernel<OUT>, mq, mk, mv, mo, ms, ml, p);
}

}  // namespace

cudaError_t launch_linear_tc_items(const LinearWork& p, bool out, int units, cudaStream_t stream) {
  const cudaError_t e = check_registers();
  if (e != cudaSuccess) return e;
  return out ? launch_items<true>(p, units, stream) : launch_items<false>(p, units, stream);
}

}  // namespace gdn
