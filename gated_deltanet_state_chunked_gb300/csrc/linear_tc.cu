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
// One CTA owns one (segment of a sequence, v-head) and walks its chunks.  Products per chunk, all
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
// so w v = h + r + m + l up to 2^-25, in five packed bf16 instructions for two values.  (Splitting the
// fp32 product into three terms costs three times the instructions, which is what bound the kernel:
// 785 us against 843 us for 64 prompts of 1556 tokens, 16/32 heads, before the other warps kept up.)
//
// Warpgroups (four warps; registers moved between them by setmaxnreg):
//   0, 1  scores to P, outputs: a thread owns a row t, group 0 the column blocks 0 and 2 of the scores
//         and the first half of the outputs, group 1 the others.  (State only: 0-3 as 2, 3.)
//   2, 3  values to A operands, quarters of 32 tokens in turn: weight, transpose (ldmatrix), split
//   4, 5  the state: a thread owns half a row of S
//   6     one warp issues QK, QS, PV, one KV, one loads the tiles two chunks ahead and stores the
//         outputs from the stage of Q that they replace
// Every hand-off is an mbarrier; every wait is bounded.
//
// A sequence longer than `seg_tokens` is cut into segments, so that a few long prompts fill the GPU:
// the segments' own states first (KV only, from zero), then their entering states
// (linear_carry_kernel), then every segment as above.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>

#include "gdn_internal.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace {

using namespace tc;
using tcp::kbf16;
using tcp::kWaitNs;

constexpr int C = 128;           // tokens per chunk
constexpr int NWARP = 28, NT = 32 * NWARP;
constexpr int kRegsLaunch = 72;  // a thread's registers at launch, and (below) in its warpgroup's role
constexpr int kRegsRows = 72, kRegsSplit = 56, kRegsState = 112, kRegsControl = 24;
static_assert(2 * kRegsRows + 2 * kRegsSplit + 2 * kRegsState + kRegsControl <= 7 * kRegsLaunch &&
              4 * kRegsSplit + 2 * kRegsState + kRegsControl <= 7 * kRegsLaunch, "what a launch holds");
constexpr uint32_t kTile = 32768, kAtom = 16384;  // 128 rows x 128 bf16: two swizzled atoms of 64 columns

// Shared memory: with outputs two stages of [Q | K | V] and the bf16 state (K-major); state only three
// stages of [K | V].  The state's tile (there: a spare one) also stages entering and final states.
template <bool OUT>
struct Lay {
  static constexpr int kStages = OUT ? 2 : 3;
  static constexpr uint32_t Q = 0, K = OUT ? 2 * kTile : 0, V = K + kStages * kTile;
  static constexpr uint32_t S = V + kStages * kTile;
  static constexpr uint32_t CF = S + kTile;        // pw(31 - j)
  static constexpr uint32_t W = CF + 4 * 32;       // weight terms, of a whole and of the last chunk
  static constexpr uint32_t BARS = W + 2 * 768;
  static constexpr uint32_t SCRATCH = BARS + 8 * 40;
  static constexpr uint32_t TOTAL = SCRATCH + 4 * 16;
  static constexpr uint32_t ALLOC = TOTAL + 1024;
  static_assert(ALLOC <= 232448, "shared memory");
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

enum Bar { kFull = 0, kEmpty = 3, kAFull = 6, kAFree = 10, kKV = 14, kKVFree = 16, kQK = 18, kP, kOFull, kOFree, kStaged,
           kSFull, kSFree, kFix, kDrainA, kDrainB, kCorner, kPair /* one per quad */, kBars = kPair + 4 };

struct TcParams {
  const float* log_decay;
  const int32_t* cu;
  const float* S0;
  float* local;  // [units][h_v][d_v][d_k]: the segments' own, then entering states
  __nv_bfloat16* O;
  float* S_out;
  int* status;
  int n_seqs, total_tokens, h_k, h_v, d_k, d_v;
  int seg_tokens;  // INT_MAX: sequences are not cut
  int skip_last;   // segment states only: the last segment of each sequence is not needed
  float scale;
};

// The work list: unit u is segment `seg` of sequence `seq`; sequences in order, those with a
// malformed range (see chunk_info_n) left out, an empty sequence one unit.
struct Unit {
  int seq, seg, n_seg, t_begin, t_end, seq_end, first;
  bool any_bad;
};
__device__ __forceinline__ int segments_of(int len, int seg_tokens) {
  return len <= seg_tokens ? 1 : (len - 1) / seg_tokens + 1;
}

// The unit `want`, or (want < 0) sequence `want_seq`'s units; seq = -1 when there is none.  The first
// warp walks the offsets, 128 at a time with the next ones under way, and stops at the unit found
// (`all`: goes on to the end, so that any_bad speaks of every range).  scratch: 8 ints.
__device__ inline Unit find_unit(const int32_t* cu, int n_seqs, int total, int seg_tokens, int want, int want_seq, bool all,
                                 int* scratch) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {
    if (lane < 8) scratch[lane] = lane == 0 ? -1 : 0;
    __syncwarp();
    int carry = 0, high = INT_MIN, next[5];
    bool found = false, bad = false;
    auto fetch = [&](int base) {
#pragma unroll
      for (int e = 0; e < 5; ++e) next[e] = base + 4 * lane + e <= n_seqs ? cu[base + 4 * lane + e] : 0;
    };
    fetch(0);
    for (int base = 0; base < n_seqs && (all || !found); base += 128) {
      int off[5];
#pragma unroll
      for (int e = 0; e < 5; ++e) off[e] = next[e];
      fetch(base + 128);
      // the largest offset before each range: this lane's, the lanes' before it, the rounds' before
      int top = INT_MIN;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (base + 4 * lane + e < n_seqs) top = max(top, max(off[e], off[e + 1]));
      int incl = top;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl = max(incl, x);
      }
      int before = __shfl_up_sync(0xffffffffu, incl, 1);
      before = lane == 0 ? high : max(high, before);
      high = max(high, __shfl_sync(0xffffffffu, incl, 31));
      int cnt[4], sum = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = base + 4 * lane + e < n_seqs;
        const bool ok = in && off[e] >= 0 && off[e] >= before && off[e + 1] >= off[e] && off[e + 1] <= total;
        if (in) before = max(before, max(off[e], off[e + 1]));
        bad |= in && !ok;
        cnt[e] = ok ? segments_of(off[e + 1] - off[e], seg_tokens) : 0;
        sum += cnt[e];
      }
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      int first = carry + inc - sum;
      bool here = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = base + 4 * lane + e;
        if (cnt[e] > 0 && (want >= 0 ? want >= first && want < first + cnt[e] : i == want_seq)) {
          here = true;
          scratch[0] = i;
          scratch[1] = want >= 0 ? want - first : 0;
          scratch[2] = cnt[e];
          scratch[3] = off[e];
          scratch[4] = off[e + 1];
          scratch[5] = first;
        }
        first += cnt[e];
      }
      found |= __any_sync(0xffffffffu, here);
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) scratch[6] = 1;
  }
  __syncthreads();
  Unit u;
  u.seq = scratch[0];
  u.seg = scratch[1];
  u.n_seg = scratch[2];
  u.seq_end = scratch[4];
  u.first = scratch[5];
  u.any_bad = scratch[6] != 0;
  u.t_begin = scratch[3] + u.seg * (u.n_seg > 1 ? seg_tokens : 0);
  u.t_end = u.seg + 1 < u.n_seg ? u.t_begin + seg_tokens : u.seq_end;
  return u;
}

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
// Packed bf16 products, rounded once.
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
// 32 lanes x 16 columns (thread i -> lane i).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
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

// OUT: outputs and the final state; otherwise the states of the units alone (to S_out when a sequence
// is one unit, to `local`, from zero, when it is cut).
template <bool OUT>
__global__ void __launch_bounds__(NT, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                     const TcParams p) {
  using L = Lay<OUT>;
  using TM = Tmem<OUT>;
  static_assert(kBars <= 40, "barrier area");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* cf = reinterpret_cast<float*>(sm + L::CF);
  uint32_t* wtab = reinterpret_cast<uint32_t*>(sm + L::W);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BARS);
  int* scratch = reinterpret_cast<int*>(sm + L::SCRATCH);
  volatile int* dead = scratch + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scratch + 9);
  int* issued = scratch + 10;  // chunks whose loads were issued

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = warp >> 2, quad = warp & 3;
  const int h = blockIdx.x % p.h_v;
  const int unit = blockIdx.x / p.h_v;
  const Unit un = find_unit(p.cu, p.n_seqs, p.total_tokens, p.seg_tokens, unit, 0, unit == 0 && h == 0, scratch);
  if (unit == 0 && h == 0 && tid == 0 && un.any_bad) atomicExch(p.status, GDN_ERR_SHAPE);
  if (un.seq < 0) return;
  if (!OUT && p.skip_last && un.seg + 1 == un.n_seg) return;  // (a sequence of one segment too)
  const int t_begin = un.t_begin, len = un.t_end - un.t_begin;
  const int n_chunks = (len + C - 1) / C;
  const int n_last = len - (n_chunks - 1) * C;  // tokens of the last chunk
  const int hk = h / (p.h_v / p.h_k);
  const int dkp = p.d_k <= 64 ? 64 : 128, dvp = p.d_v <= 64 ? 64 : 128;  // columns that the products cover
  const float g = p.log_decay[h];

  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int b = 0; b < kBars; ++b) {
      int count = 1;
      if (b >= kEmpty && b < kEmpty + 3) count = OUT ? 2 : 1;  // the issuing warps' commits
      if (b >= kAFull && b < kAFull + 4) count = 4;             // the warps of a splitting group
      if (b == kP || b == kOFree || b == kStaged || b == kSFull || b == kKVFree || b == kKVFree + 1 || b == kFix || b == kCorner) count = 8;
      if (b >= kPair) count = 2;
      mbar_init(&bar[b], count);
    }
    mbar_fence_init();
    *dead = 0;
    *issued = 0;
  }
  if (tid < 32) cf[tid] = tid == 31 ? 1.f : expf((float)(31 - tid) * g);
  // Weight terms: word 12 (4 q + j) + 4 term + e holds those of tokens 32 q + 8 e + 2 j + {0, 1}; the
  // second table those of the last chunk, zero behind its end.
  if (tid >= 64 && tid < 64 + 128) {
    const int i = tid - 64, which = i >> 6, q = (i >> 4) & 3, j = (i >> 2) & 3, e = i & 3;
    const int n = which ? n_last : C;
    uint32_t term[3] = {0u, 0u, 0u};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int back = n - 1 - (32 * q + 8 * e + 2 * j + x);
      float w = back < 0 ? 0.f : back == 0 ? 1.f : expf((float)back * g);
#pragma unroll
      for (int y = 0; y < 3; ++y) {
        const uint32_t b = __float_as_uint(w) & 0xffff0000u;
        w -= __uint_as_float(b);
        term[y] |= x ? b : b >> 16;
      }
    }
#pragma unroll
    for (int y = 0; y < 3; ++y) wtab[192 * which + 12 * (4 * q + j) + 4 * y + e] = term[y];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
  auto wait = [&](int b, int parity) {
    if (mbar_wait(&bar[b], (uint32_t)(parity & 1), kWaitNs)) return true;
    *dead = 1;
    return false;
  };
  auto arrive = [&](int b) {  // one arrival per warp, behind what its threads did before
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[b]);
  };

  if (OUT && group < 2) {
    // ------------------------------------------------------------ scores to P, outputs
    const int t = 32 * quad + lane;
    const float rho = fmaxf(expf((float)(t + 1) * g), 8.673617379884035e-19f);  // 2^-60
    const float inv = 1.f / rho, f = rho * p.scale;
    // The factor of a score is lambda^(t - s) / rho_t = rf cf[j] for column j of a block: rf =
    // lambda^(t - 32 b - 31) / rho_t, and cf[j] = lambda^(31 - j).  On the diagonal (t - 32 b = lane)
    // rf's power has a negative exponent; where rf could leave the fp32 range (a decay below e^-1.4 per
    // token) the block takes cf[31 - lane + j] instead.
    const bool steep = !(cf[0] > 1e-19f);
    float rf[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int b = 2 * i + group;
      rf[i] = b < quad ? expf((float)(t - 32 * b - 31) * g) * inv : steep ? inv : inv / cf[lane];
    }
    for (int c = 0; c < n_chunks; ++c) {
      const int n = c + 1 < n_chunks ? C : n_last;
      if (!wait(kQK, c)) break;
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
          if (b < quad || !steep) {
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
      if (!wait(kPair + quad, c)) break;
      tmem_st16(tmem + lane_base + TM::cP + 16 * group, o[0]);
      tmem_st16(tmem + lane_base + TM::cP + 32 + 16 * group, o[1]);
      tmem_st_wait();
      tc_fence_before();
      arrive(kP);
      if (!wait(kOFull, c)) break;
      tc_fence_after();
      // The outputs, rounded, into the stage of Q (whose readers are done)
      unsigned char* stage = sm + L::Q + (c & 1) * kTile;
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
      if (n == C) {
        fence_async_smem();
        arrive(kStaged);
      } else if (8 * (lane & 7) + 64 * group < p.d_v) {
        // a part of a chunk: the rows behind its end are not this sequence's
        const int col = 64 * group + 8 * (lane & 7);
        for (int row = 32 * quad + (lane >> 3); row < min(n, 32 * quad + 32); row += 4)
          *reinterpret_cast<uint4*>(p.O + ((size_t)(t_begin + c * C + row) * p.h_v + h) * p.d_v + col) =
              *reinterpret_cast<const uint4*>(stage + kbf16(row, col, 128));
      }
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
    for (int c = 0; c < n_chunks && ok; ++c) {
      const int st = c % L::kStages, n = c + 1 < n_chunks ? C : n_last;
      if (!(ok = wait(kFull + st, c / L::kStages))) break;
      const uint32_t* table = wtab + (n == C ? 0 : 192) + 12 * (lane & 3);
#pragma unroll 1
      for (int i = 0; i < kPer; ++i) {
        const int q = buf + TM::kABufs * i, m = c * kPer + i;
        uint32_t x[4][4];  // tiles of 16 rows x 16 tokens: (rows +0, tokens +0), (+0, +16), (+16, +0), (+16, +16)
        uint32_t wt[3][4];
        if (rows) {
          const uint32_t vt = smem_u32(sm + L::V + st * kTile) + (uint32_t)(32 * q + lm_tok) * 128u;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int d = lm_d + 16 * (b >> 1);
            ldmatrix_x4_trans(vt + (d >> 6) * kAtom + 2048 * (b & 1) + ((((d & 63) >> 3) ^ (lm_tok & 7)) << 4), x[b]);
          }
#pragma unroll
          for (int y = 0; y < 3; ++y) {
            const uint4 u = *reinterpret_cast<const uint4*>(table + 48 * q + 4 * y);
            wt[y][0] = u.x; wt[y][1] = u.y; wt[y][2] = u.z; wt[y][3] = u.w;
          }
          if (n < C) {  // (a row behind the last token may hold anything)
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int tok = 32 * q + 16 * (b & 1) + 8 * (j >> 1) + 2 * (lane & 3);
                x[b][j] = tok >= n ? 0u : tok + 1 >= n ? x[b][j] & 0xffffu : x[b][j];
              }
          }
        }
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
              t[1][j] = bfma2(v, w[0], t[0][j] ^ 0x80008000u);
              t[2][j] = bmul2(v, w[4]);
              t[3][j] = bfma2(v, w[8], bfma2(v, w[4], t[2][j] ^ 0x80008000u));
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
  } else if (group < 6) {
    // ------------------------------------------------------------ the state
    regs_inc<kRegsState>();
    const int hw = group - 4;
    const int r = 32 * quad + lane;  // row of S
    const bool mine = 32 * quad < dvp && 64 * hw < dkp;
    float s[64];
    const float* S_in = nullptr;
    if (un.n_seg == 1) {
      if (p.S0) S_in = p.S0 + ((size_t)un.seq * p.h_v + h) * p.d_v * p.d_k;
    } else if (OUT) {
      S_in = p.local + ((size_t)unit * p.h_v + h) * p.d_v * p.d_k;
    }
    // Entering and final states pass through a corner of the state's tile, 32 rows x 32 columns per warp
    // (16-byte chunks swizzled by row), so that global memory sees whole 128-byte lines.
    float* corner = reinterpret_cast<float*>(sm + L::S) + 1024 * (warp - 16);
    const int my_chunk = lane & 7, my_row = lane >> 3;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = 64 * hw + 32 * j + 4 * my_chunk;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = 4 * i + my_row;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (S_in && 32 * quad + row < p.d_v && k < p.d_k)
          x = *reinterpret_cast<const float4*>(S_in + (size_t)(32 * quad + row) * p.d_k + k);
        *reinterpret_cast<float4*>(corner + 32 * row + 4 * (my_chunk ^ (row & 7))) = x;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(corner + 32 * lane + 4 * (i ^ (lane & 7)));
        s[32 * j + 4 * i] = x.x; s[32 * j + 4 * i + 1] = x.y; s[32 * j + 4 * i + 2] = x.z; s[32 * j + 4 * i + 3] = x.w;
      }
    }
    // (the rounded state that follows is written over other warps' corners)
    arrive(kCorner);
    if (!wait(kCorner, 0)) s[0] = 0.f;
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
    if (OUT && n_chunks > 0) publish_state();
    const DecayStep step = decay_step(g, C);
    bool ok = true;
    for (int c = 0; c < n_chunks && ok; ++c) {
      const int st = c % L::kStages, kv = c % TM::kKVBufs, n = c + 1 < n_chunks ? C : n_last;
      if (n < C) {
        // rows behind the last token: another sequence's, or none; they may hold anything
        if (!(ok = wait(kFull + st, c / L::kStages))) break;
        const int per_row = (dkp + dvp) / 8;
        for (int e = tid - 512; e < (C - n) * per_row; e += 256) {
          const int row = n + e / per_row, x = e % per_row;
          unsigned char* tile = x < dkp / 8 ? sm + L::K + st * kTile : sm + L::V + st * kTile;
          const int col = x < dkp / 8 ? x : x - dkp / 8;
          *reinterpret_cast<uint4*>(tile + (col >> 3) * kAtom + row * 128 + (col & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_smem();
        arrive(kFix);
      }
      if (!(ok = wait(kKV + kv, c / TM::kKVBufs))) break;
      tc_fence_after();
      const DecayStep f = n == C ? step : decay_step(g, n);
      if (mine) {
        const uint32_t at = tmem + lane_base + TM::cKV + 128 * kv + 64 * hw;
        const uint64_t m = f.near1 ? pair(f.f1, f.f1) : pair(f.f, f.f);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float x[32];
          tmem_ld32(at + 32 * b, x);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float &s0 = s[32 * b + j], &s1 = s[32 * b + j + 1];
            const uint64_t d = pair(x[j], x[j + 1]), a = pair(s0, s1);
            unpair(fma2(a, m, f.near1 ? add2(a, d) : d), s0, s1);
          }
        }
      }
      tc_fence_before();
      arrive(kKVFree + kv);
      if (OUT && c + 1 < n_chunks) {
        if (!(ok = wait(kSFree, c))) break;
        publish_state();
      }
    }
    float* dst = nullptr;
    if (un.n_seg == 1 || (OUT && un.seg + 1 == un.n_seg))
      dst = p.S_out + ((size_t)un.seq * p.h_v + h) * p.d_v * p.d_k;
    else if (!OUT)
      dst = p.local + ((size_t)unit * p.h_v + h) * p.d_v * p.d_k;
    // (the last reader of the state's tile, QS of the last chunk, must be done with it)
    if (OUT && ok && n_chunks > 0) ok = wait(kSFree, n_chunks - 1);
    if (dst && ok) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = 64 * hw + 32 * j + 4 * my_chunk;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(corner + 32 * lane + 4 * (i ^ (lane & 7))) =
              make_float4(s[32 * j + 4 * i], s[32 * j + 4 * i + 1], s[32 * j + 4 * i + 2], s[32 * j + 4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = 4 * i + my_row;
          if (32 * quad + row < p.d_v && k < p.d_k)
            *reinterpret_cast<float4*>(dst + (size_t)(32 * quad + row) * p.d_k + k) =
                *reinterpret_cast<const float4*>(corner + 32 * row + 4 * (my_chunk ^ (row & 7)));
        }
      }
    }
  } else {
    regs_dec<kRegsControl>();
    if (quad == 0) {
      // ---------------------------------------------------------- QK, QS, PV
      if constexpr (OUT) {
        const uint32_t idQK = idesc_bf16(128, 128, false, false), idQS = idesc_bf16(128, dvp, false, false),
                       idPV = idesc_bf16(128, dvp, false, true);
        const int nk = (p.d_k + 15) / 16;
        const uint64_t dS = sdesc_sw128(smem_u32(sm + L::S), 16, 1024);
        auto issue_qk = [&](int c) {
          if (!wait(kFull + (c & 1), c >> 1)) return false;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t dQ = sdesc_sw128(smem_u32(sm + L::Q + (c & 1) * kTile), 16, 1024);
            const uint64_t dK = sdesc_sw128(smem_u32(sm + L::K + (c & 1) * kTile), 16, 1024);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < nk) {
                const uint64_t off = (uint64_t)(((k >> 2) * kAtom + (k & 3) * 32) >> 4);
                mma_bf16(tmem + TM::cP, dQ + off, dK + off, idQK, k > 0);
              }
            mma_commit(&bar[kQK]);
          }
          __syncwarp();
          return true;
        };
        if (n_chunks > 0 && issue_qk(0)) {
          for (int c = 0; c < n_chunks; ++c) {
            const int st = c % L::kStages;
            if (!wait(kSFull, c)) break;
            if (c > 0 && !wait(kOFree, c - 1)) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t dQ = sdesc_sw128(smem_u32(sm + L::Q + st * kTile), 16, 1024);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (k < nk) {
                  const uint64_t off = (uint64_t)(((k >> 2) * kAtom + (k & 3) * 32) >> 4);
                  mma_bf16(tmem + TM::cO, dQ + off, dS + off, idQS, k > 0);
                }
              mma_commit(&bar[kSFree]);
            }
            __syncwarp();
            if (!wait(kP, c)) break;
            if (c + 1 == n_chunks && n_last < C && !wait(kFix, 0)) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t dV = sdesc_sw128(smem_u32(sm + L::V + st * kTile), kAtom, 1024);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mma_bf16_ts(tmem + TM::cO, tmem + TM::cP + 8 * k, dV + (uint64_t)((k * 2048) >> 4), idPV, 1);
              mma_commit(&bar[kOFull]);
              mma_commit(&bar[kEmpty + st]);
            }
            __syncwarp();
            if (c + 1 < n_chunks && !issue_qk(c + 1)) break;
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
      for (int c = 0; c < n_chunks && ok; ++c) {
        const int st = c % L::kStages, kv = c % TM::kKVBufs;
        const uint32_t d = tmem + TM::cKV + 128 * kv;
        if (!(ok = wait(kFull + st, c / L::kStages))) break;
        if (c + 1 == n_chunks && n_last < C && !(ok = wait(kFix, 0))) break;
        if (c >= TM::kKVBufs && !(ok = wait(kKVFree + kv, c / TM::kKVBufs - 1))) break;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          const int buf = q % TM::kABufs, m = c * (4 / TM::kABufs) + q / TM::kABufs;
          if (!(ok = wait(kAFull + buf, m))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t dK = sdesc_sw128(smem_u32(sm + L::K + st * kTile), kAtom, 1024);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint64_t b = dK + (uint64_t)(((32 * q + 16 * k) * 128) >> 4);
              const uint32_t a = tmem + TM::cA + buf * TM::ASTEP + 8 * k;
              mma_bf16_ts(d, a + 48, b, idKV, q > 0 || k > 0);
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
      auto store = [&](int c) {  // chunk c's outputs out of its stage of Q, which is then free
        if (!wait(kStaged, c)) return false;
        if (lane == 0) {
          for (int x = 0; x < dvp; x += 64)
            tma_store_3d(&map_o, sm + L::Q + (c & 1) * kTile + (x >> 6) * kAtom, x, h, t_begin + c * C);
          bulk_commit();
          bulk_wait_read_all();
        }
        __syncwarp();
        return true;
      };
      bool ok = true;
      for (int c = 0; c < n_chunks; ++c) {
        const int st = c % L::kStages, t0 = t_begin + c * C;
        if (c >= L::kStages && !(ok = wait(kEmpty + st, c / L::kStages - 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar[kFull + st], bytes);
          for (int x = 0; x < dkp; x += 64)
            tma_load_3d(sm + L::K + st * kTile + (x >> 6) * kAtom, &map_k, &bar[kFull + st], x, hk, t0);
          for (int x = 0; x < dvp; x += 64)
            tma_load_3d(sm + L::V + st * kTile + (x >> 6) * kAtom, &map_v, &bar[kFull + st], x, h, t0);
        }
        __syncwarp();
        if (OUT) {
          const bool stored = c < 2 || (ok = store(c - 2));
          if (lane == 0) {  // (loaded all the same, so that the stage's bytes are whole when a wait gave up)
            for (int x = 0; x < dkp; x += 64)
              tma_load_3d(sm + L::Q + st * kTile + (x >> 6) * kAtom, &map_q, &bar[kFull + st], x, hk, t0);
          }
          if (!stored) {
            if (lane == 0) *issued = c + 1;
            break;
          }
        }
        if (lane == 0) *issued = c + 1;
        __syncwarp();
      }
      if (OUT && ok)
        for (int c = max(0, n_chunks - 2); c < n_chunks; ++c)
          if ((c + 1 < n_chunks || n_last == C) && !store(c)) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*dead) {
    // A wait gave up: let the loads in flight land (each wait bounded; the MMAs were drained by their
    // issuing warps), then report.  The results are unspecified.
    if (tid == 0) {
      for (int c = max(0, *issued - L::kStages); c < *issued; ++c)
        mbar_wait(&bar[kFull + c % L::kStages], (uint32_t)((c / L::kStages) & 1), kWaitNs);
      atomicExch(p.status, GDN_ERR_TIMEOUT);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// The entering states of a cut sequence's segments, in place of the segments' own states, and (FINAL)
// the state behind the last one.  Element by element: E <- lambda^seg E + local.
constexpr int kCarryNT = 256;
template <bool FINAL>
__global__ void __launch_bounds__(kCarryNT) linear_carry_kernel(const TcParams p) {
  __shared__ int scratch[8];
  const int h = blockIdx.x % p.h_v, seq = blockIdx.x / p.h_v;
  const Unit un = find_unit(p.cu, p.n_seqs, p.total_tokens, p.seg_tokens, -1, seq, false, scratch);
  if (un.seq < 0 || un.n_seg == 1) return;
  const float g = p.log_decay[h];
  const int dd = p.d_v * p.d_k;
  const int e = (blockIdx.y * kCarryNT + threadIdx.x) * 4;
  if (e >= dd) return;
  const size_t at = ((size_t)seq * p.h_v + h) * dd + e;
  float4 E = p.S0 ? *reinterpret_cast<const float4*>(p.S0 + at) : make_float4(0.f, 0.f, 0.f, 0.f);
  const DecayStep step = decay_step(g, p.seg_tokens);
  const size_t stride = (size_t)p.h_v * dd;
  float* loc = p.local + ((size_t)un.first * p.h_v + h) * dd + e;
  for (int j = 0; j < un.n_seg; ++j, loc += stride) {
    const bool last = j + 1 == un.n_seg;
    if (FINAL || !last) {
      const float4 x = *reinterpret_cast<const float4*>(loc);
      if (!FINAL) *reinterpret_cast<float4*>(loc) = E;
      const DecayStep f = last ? decay_step(g, un.seq_end - (un.t_begin + j * p.seg_tokens)) : step;
      E = make_float4(f(E.x, x.x), f(E.y, x.y), f(E.z, x.z), f(E.w, x.w));
    } else {
      *reinterpret_cast<float4*>(loc) = E;
    }
  }
  if (FINAL) *reinterpret_cast<float4*>(p.S_out + at) = E;
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

int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    sms = 152;
  return sms;
}

constexpr int kMinSegment = 512;

// Tokens per segment: one sequence's segments times the v-heads fill the GPU once.
int segment_tokens(int total_tokens, int h_v) {
  const int parts = std::max(1, device_sms() / h_v);
  const int seg = ((total_tokens + parts - 1) / parts + C - 1) / C * C;
  return seg >= total_tokens ? INT_MAX : std::max(seg, kMinSegment);
}

}  // namespace

bool linear_tc_supported(const LinearParams& p) { return p.total_tokens > 0; }

size_t linear_tc_workspace_bytes(const LinearParams& p) {
  const int seg = segment_tokens(p.total_tokens, p.h_v);
  if (seg >= p.total_tokens) return 0;
  return ((size_t)p.n_seqs + p.total_tokens / seg) * p.h_v * p.d_v * p.d_k * 4;
}

cudaError_t launch_linear_tc(const LinearParams& lp, void* workspace, cudaStream_t stream) {
  CUtensorMap mq{}, mk, mv, mo{};
  if ((lp.write_O && (!make_map_heads(&mq, lp.q, lp.total_tokens, lp.h_k, lp.d_k) ||
                      !make_map_heads(&mo, lp.O, lp.total_tokens, lp.h_v, lp.d_v))) ||
      !make_map_heads(&mk, lp.k, lp.total_tokens, lp.h_k, lp.d_k) ||
      !make_map_heads(&mv, lp.v, lp.total_tokens, lp.h_v, lp.d_v))
    return cudaErrorInvalidValue;
  TcParams p{};
  p.log_decay = lp.log_decay; p.cu = lp.cu; p.S0 = lp.S0; p.local = static_cast<float*>(workspace);
  p.O = static_cast<__nv_bfloat16*>(lp.O); p.S_out = lp.S_out; p.status = lp.status;
  p.n_seqs = lp.n_seqs; p.total_tokens = lp.total_tokens; p.h_k = lp.h_k; p.h_v = lp.h_v; p.d_k = lp.d_k; p.d_v = lp.d_v;
  p.scale = lp.scale;
  const int seg = segment_tokens(lp.total_tokens, lp.h_v);
  const bool cut = seg < lp.total_tokens;
  p.seg_tokens = cut ? seg : INT_MAX;
  p.skip_last = cut && lp.write_O;
  const long long units = (long long)lp.n_seqs + (cut ? lp.total_tokens / seg : 0);
  const long long blocks = units * lp.h_v;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<true>::ALLOC);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(linear_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<false>::ALLOC);
  if (e != cudaSuccess) return e;
  // (the warpgroups' shares add up to what the kernel is launched with: a smaller launch would wait)
  cudaFuncAttributes attr;
  for (const void* k : {reinterpret_cast<const void*>(linear_tc_kernel<true>), reinterpret_cast<const void*>(linear_tc_kernel<false>)}) {
    e = cudaFuncGetAttributes(&attr, k);
    if (e != cudaSuccess) return e;
    if (attr.numRegs != kRegsLaunch) return cudaErrorInvalidKernelImage;
  }
  if (cut || !lp.write_O) {
    linear_tc_kernel<false><<<(unsigned)blocks, NT, Lay<false>::ALLOC, stream>>>(mq, mk, mv, mo, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (cut) {
    const dim3 grid((unsigned)((long long)lp.n_seqs * lp.h_v), (lp.d_v * lp.d_k / 4 + kCarryNT - 1) / kCarryNT);
    if (lp.write_O) linear_carry_kernel<false><<<grid, kCarryNT, 0, stream>>>(p);
    else linear_carry_kernel<true><<<grid, kCarryNT, 0, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (lp.write_O) {
    linear_tc_kernel<true><<<(unsigned)blocks, NT, Lay<true>::ALLOC, stream>>>(mq, mk, mv, mo, p);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace gdn
