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
//   KV   (W V)^T K         A = the decay-weighted values, transposed, as three bf16 terms (hi, mid,
//                          lo: 24 bits, so that the state keeps fp32 accuracy) in TMEM, B = K    24
// O's operands S and P are rounded once each, as the output itself is; the state is carried in fp32
// registers and never read back from its rounded copy.
//
// Warps: 0-3 turn QK into P and write the outputs (a thread owns a row t); 4-11 weight, transpose
// (ldmatrix) and split the values in quarters of 32 tokens, and carry the state (a thread owns half a
// row of S); 12 issues QK, QS, PV; 13 issues KV; 14 loads the tiles two chunks ahead.  Every hand-off
// is an mbarrier; every wait is bounded.
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
constexpr int NWARP = 15, NT = 32 * NWARP;
constexpr uint32_t kTile = 32768, kAtom = 16384;  // 128 rows x 128 bf16: two swizzled atoms of 64 columns

struct Lay {
  static constexpr uint32_t Q = 0, K = 2 * kTile, V = 4 * kTile;  // two stages each
  static constexpr uint32_t S = 6 * kTile;                        // bf16 state, K-major
  static constexpr uint32_t PW = 7 * kTile;                       // 32 zeros, pw(0..128)
  static constexpr uint32_t CF = PW + 4 * 164;                    // pw(31 - j)
  static constexpr uint32_t BARS = CF + 4 * 32;
  static constexpr uint32_t SCRATCH = BARS + 8 * 24;
  static constexpr uint32_t TOTAL = SCRATCH + 4 * 48;
  static constexpr uint32_t ALLOC = TOTAL + 1024;
  static_assert(ALLOC <= 232448, "shared memory");
  // TMEM columns: QK (then P), O, KV, two buffers of [hi | mid | lo] for 32 tokens
  static constexpr uint32_t cP = 0, cO = 128, cKV = 256, cA = 384;
  static constexpr uint32_t ASTEP = 48;
};

enum Bar { kFull = 0, kEmpty = 2, kAFull = 4, kAFree = 6, kQK = 8, kP, kOFull, kOFree, kSFull, kSFree, kKV, kKVFree, kFix,
           kDrainA, kDrainB, kBars };
static_assert(kBars <= 24, "barrier area");

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

// Block-wide over NW warps: the unit `want`, or (want < 0) sequence `want_seq`'s units.  seq = -1 when
// there is none.  scratch: 2 NW + 8 ints.
template <int NW>
__device__ inline Unit find_unit(const int32_t* cu, int n_seqs, int total, int seg_tokens, int want, int want_seq,
                                 int* scratch) {
  constexpr int NTH = 32 * NW, RS = 2 * NW;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 8) scratch[RS + tid] = tid == 0 ? -1 : 0;
  __syncthreads();
  int carry = 0, carry_max = cu[0];
  for (int base = 0; base < n_seqs; base += NTH) {
    const int i = base + tid;
    int a = 0, b = INT_MIN;
    if (i < n_seqs) { a = cu[i]; b = cu[i + 1]; }
    int incl = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl = max(incl, x);
    }
    int excl = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) excl = INT_MIN;
    if (lane == 31) scratch[NW + warp] = incl;
    __syncthreads();
    int wmax = INT_MIN, allmax = INT_MIN;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int m = scratch[NW + w];
      if (w < warp) wmax = max(wmax, m);
      allmax = max(allmax, m);
    }
    const int before = max(carry_max, max(wmax, excl));
    const bool ok = i < n_seqs && a >= 0 && a >= before && b >= a && b <= total;
    const int cnt = ok ? segments_of(b - a, seg_tokens) : 0;
    int inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    int wsum = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int s = scratch[w];
      if (w < warp) wsum += s;
      all += s;
    }
    const int ex = carry + wsum + inc - cnt;
    if (i < n_seqs && !ok) scratch[RS + 6] = 1;
    if (cnt > 0 && (want >= 0 ? want >= ex && want < ex + cnt : i == want_seq)) {
      scratch[RS] = i;
      scratch[RS + 1] = want >= 0 ? want - ex : 0;
      scratch[RS + 2] = cnt;
      scratch[RS + 3] = a;
      scratch[RS + 4] = b;
      scratch[RS + 5] = ex;
    }
    carry += all;
    carry_max = max(carry_max, allmax);
    __syncthreads();
  }
  Unit u;
  u.seq = scratch[RS];
  u.seg = scratch[RS + 1];
  u.n_seg = scratch[RS + 2];
  u.seq_end = scratch[RS + 4];
  u.first = scratch[RS + 5];
  u.any_bad = scratch[RS + 6] != 0;
  u.t_begin = scratch[RS + 3] + u.seg * (u.n_seg > 1 ? seg_tokens : 0);
  u.t_end = u.seg + 1 < u.n_seg ? u.t_begin + seg_tokens : u.seq_end;
  __syncthreads();
  return u;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

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
// 16 TMEM lanes x 8 columns: registers 0 and 1 are rows lane / 4 and lane / 4 + 8 of columns
// lane % 4, registers 2 and 3 the same rows of columns 4 + lane % 4.
__device__ __forceinline__ void tmem_st_16x128b_x2(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
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

// OUT: outputs and the final state; otherwise the states of the units alone (to S_out when a sequence
// is one unit, to `local`, from zero, when it is cut).
template <bool OUT>
__global__ void __launch_bounds__(NT, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const TcParams p) {
  using L = Lay;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* pwz = reinterpret_cast<float*>(sm + L::PW);
  float* pw = pwz + 32;  // pw[n] = lambda^n, zero at negative n
  float* cf = reinterpret_cast<float*>(sm + L::CF);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BARS);
  int* scratch = reinterpret_cast<int*>(sm + L::SCRATCH);
  volatile int* dead = scratch + 40;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scratch + 41);
  int* issued = scratch + 42;  // chunks whose loads were issued

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.h_v;
  const int unit = blockIdx.x / p.h_v;
  const Unit un = find_unit<NWARP>(p.cu, p.n_seqs, p.total_tokens, p.seg_tokens, unit, 0, scratch);
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
      const int count = b == kEmpty || b == kEmpty + 1 ? (OUT ? 2 : 1)
                        : b == kP || b == kOFree       ? 4
                        : b == kAFull || b == kAFull + 1 || b == kSFull || b == kKVFree || b == kFix ? 8 : 1;
      mbar_init(&bar[b], count);
    }
    mbar_fence_init();
    *dead = 0;
    *issued = 0;
  }
  for (int n = tid; n < 32 + C + 1; n += NT) pwz[n] = n < 32 ? 0.f : n == 32 ? 1.f : expf((float)(n - 32) * g);
  if (tid < 32) cf[tid] = tid == 31 ? 1.f : expf((float)(31 - tid) * g);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](int b, int parity) {
    if (mbar_wait(&bar[b], (uint32_t)(parity & 1), kWaitNs)) return true;
    *dead = 1;
    return false;
  };

  if (warp < 4) {
    // ------------------------------------------------------------ scores to P, outputs
    if constexpr (OUT) {
      const int quad = warp, t = 32 * quad + lane;
      const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
      const float rho = fmaxf(pw[t + 1], 8.673617379884035e-19f);  // 2^-60
      const float inv = 1.f / rho;
      for (int c = 0; c < n_chunks; ++c) {
        const int n = c + 1 < n_chunks ? C : n_last;
        if (!wait(kQK, c)) break;
        tc_fence_after();
        // blocks of 32 columns: all of the row's tokens before `quad`, none behind it
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          uint32_t o[16];
          if (b <= quad) {
            float x[32];
            tmem_ld32(tmem + lane_base + L::cP + 32 * b, x);
            tmem_ld_wait();
            if (b < quad) {
              const float rf = pw[t - 32 * b - 31] * inv;
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(cf + j);
                o[j / 2] = pack_bf16(x[j] * (rf * f.x), x[j + 1] * (rf * f.y));
                o[j / 2 + 1] = pack_bf16(x[j + 2] * (rf * f.z), x[j + 3] * (rf * f.w));
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const float y0 = j <= lane ? x[j] * (pw[lane - j] * inv) : 0.f;
                const float y1 = j + 1 <= lane ? x[j + 1] * (pw[lane - j - 1] * inv) : 0.f;
                o[j / 2] = pack_bf16(y0, y1);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = 0u;
          }
          // (P's columns [16 b, 16 b + 16) hold scores of blocks already read)
          tmem_st16(tmem + lane_base + L::cP + 16 * b, o);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kP]);
        if (!wait(kOFull, c)) break;
        tc_fence_after();
        const float f = rho * p.scale;
        uint32_t o[64];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (32 * b < dvp) {
            float x[32];
            tmem_ld32(tmem + lane_base + L::cO + 32 * b, x);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 2) o[16 * b + j / 2] = pack_bf16(f * x[j], f * x[j + 1]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kOFree]);
        if (t < n) {
          uint4* dst = reinterpret_cast<uint4*>(p.O + ((size_t)(t_begin + c * C + t) * p.h_v + h) * p.d_v);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (8 * j < p.d_v) dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ values to A operands, the state
    const int w2 = warp - 4, quad = w2 & 3, hw = w2 >> 2;
    const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
    const int r = 32 * quad + lane;  // row of S
    const bool rows = 32 * quad < dvp, cols = 64 * hw < dkp;
    float s[64];
    const float* S_in = nullptr;
    if (un.n_seg == 1) {
      if (p.S0) S_in = p.S0 + ((size_t)un.seq * p.h_v + h) * p.d_v * p.d_k;
    } else if (OUT) {
      S_in = p.local + ((size_t)unit * p.h_v + h) * p.d_v * p.d_k;
    }
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
      const int k = 64 * hw + j;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (S_in && r < p.d_v && k < p.d_k) x = *reinterpret_cast<const float4*>(S_in + (size_t)r * p.d_k + k);
      s[j] = x.x; s[j + 1] = x.y; s[j + 2] = x.z; s[j + 3] = x.w;
    }
    auto publish_state = [&]() {  // the state, rounded to bf16, as QS's B operand
      if (rows && cols) {
#pragma unroll
        for (int j = 0; j < 64; j += 8)
          *reinterpret_cast<uint4*>(sm + L::S + kbf16(r, 64 * hw + j, 128)) =
              make_uint4(pack_bf16(s[j], s[j + 1]), pack_bf16(s[j + 2], s[j + 3]), pack_bf16(s[j + 4], s[j + 5]),
                         pack_bf16(s[j + 6], s[j + 7]));
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[kSFull]);
    };
    if (OUT && n_chunks > 0) publish_state();
    const DecayStep step = decay_step(g, C);
    // this lane's part of the ldmatrix addresses: tile lane / 8 of (8 d) x (8 tokens), token lane % 8
    const int lm_tok = 16 * hw + (lane & 7) + 8 * (lane >> 4), lm_d = 8 * ((lane >> 3) & 1);
    bool ok = true;
    for (int c = 0; c < n_chunks && ok; ++c) {
      const int st = c & 1, n = c + 1 < n_chunks ? C : n_last;
      if (!(ok = wait(kFull + st, c >> 1))) break;
      if (n < C) {
        // rows behind the last token: another sequence's, or none; they may hold anything
        const int per_row = (dkp + dvp) / 8;
        for (int e = tid - 128; e < (C - n) * per_row; e += 256) {
          const int row = n + e / per_row, x = e % per_row;
          unsigned char* tile = x < dkp / 8 ? sm + L::K + st * kTile : sm + L::V + st * kTile;
          const int col = x < dkp / 8 ? x : x - dkp / 8;
          *reinterpret_cast<uint4*>(tile + (col >> 3) * kAtom + row * 128 + (col & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kFix]);
      }
      const uint32_t vt = smem_u32(sm + L::V + st * kTile);
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const int u = 4 * c + q, buf = u & 1;
        if (u >= 2 && !(ok = wait(kAFree + buf, (u >> 1) - 1))) break;
        tc_fence_after();
        if (rows) {
          // weights of this thread's tokens: two in registers 0 and 1, two in registers 2 and 3
          const int s0 = 32 * q + 16 * hw + 2 * (lane & 3);
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = s0 + (e & 1) + 8 * (e >> 1);
            w[e] = tok < n ? pw[n - 1 - tok] : 0.f;
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int d = 32 * quad + 16 * half + lm_d, tok = 32 * q + lm_tok;
            uint32_t x[4], hi[4], mid[4], lo[4];
            ldmatrix_x4_trans(vt + (d >> 6) * kAtom + tok * 128 + ((((d & 63) >> 3) ^ (tok & 7)) << 4), x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = i & 2;
              float a = bf_lo(x[i]) * w[e], b = bf_hi(x[i]) * w[e + 1];
              if (n < C) {  // (a masked value may be NaN until its row is cleared)
                a = s0 + 4 * e < n ? a : 0.f;
                b = s0 + 4 * e + 1 < n ? b : 0.f;
              }
              hi[i] = pack_bf16(a, b);
              a -= bf_lo(hi[i]);
              b -= bf_hi(hi[i]);
              mid[i] = pack_bf16(a, b);
              a -= bf_lo(mid[i]);
              b -= bf_hi(mid[i]);
              lo[i] = pack_bf16(a, b);
            }
            const uint32_t at = tmem + lane_base + ((uint32_t)(16 * half) << 16) + L::cA + buf * L::ASTEP + 8 * hw;
            tmem_st_16x128b_x2(at, hi);
            tmem_st_16x128b_x2(at + 16, mid);
            tmem_st_16x128b_x2(at + 32, lo);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kAFull + buf]);
      }
      if (!ok || !(ok = wait(kKV, c))) break;
      tc_fence_after();
      const DecayStep f = n == C ? step : decay_step(g, n);
      if (rows && cols) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float x[32];
          tmem_ld32(tmem + lane_base + L::cKV + 64 * hw + 32 * b, x);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) s[32 * b + j] = f(s[32 * b + j], x[j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[kKVFree]);
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
    if (dst && r < p.d_v && ok) {
#pragma unroll
      for (int j = 0; j < 64; j += 4) {
        const int k = 64 * hw + j;
        if (k < p.d_k)
          *reinterpret_cast<float4*>(dst + (size_t)r * p.d_k + k) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
      }
    }
  } else if (warp == 12) {
    // ------------------------------------------------------------ QK, QS, PV
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
              mma_bf16(tmem + L::cP, dQ + off, dK + off, idQK, k > 0);
            }
          mma_commit(&bar[kQK]);
        }
        __syncwarp();
        return true;
      };
      if (n_chunks > 0 && issue_qk(0)) {
        for (int c = 0; c < n_chunks; ++c) {
          const int st = c & 1;
          if (!wait(kSFull, c)) break;
          if (c > 0 && !wait(kOFree, c - 1)) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t dQ = sdesc_sw128(smem_u32(sm + L::Q + st * kTile), 16, 1024);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < nk) {
                const uint64_t off = (uint64_t)(((k >> 2) * kAtom + (k & 3) * 32) >> 4);
                mma_bf16(tmem + L::cO, dQ + off, dS + off, idQS, k > 0);
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
              mma_bf16_ts(tmem + L::cO, tmem + L::cP + 8 * k, dV + (uint64_t)((k * 2048) >> 4), idPV, 1);
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
  } else if (warp == 13) {
    // ------------------------------------------------------------ KV
    const uint32_t idKV = idesc_bf16(128, dkp, false, true);
    bool ok = true;
    for (int c = 0; c < n_chunks && ok; ++c) {
      const int st = c & 1;
      if (!(ok = wait(kFull + st, c >> 1))) break;
      if (c > 0 && !(ok = wait(kKVFree, c - 1))) break;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const int u = 4 * c + q, buf = u & 1;
        if (!(ok = wait(kAFull + buf, u >> 1))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t dK = sdesc_sw128(smem_u32(sm + L::K + st * kTile), kAtom, 1024);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint64_t b = dK + (uint64_t)(((32 * q + 16 * k) * 128) >> 4);
            const uint32_t a = tmem + L::cA + buf * L::ASTEP + 8 * k;
            mma_bf16_ts(tmem + L::cKV, a + 32, b, idKV, q > 0 || k > 0);
            mma_bf16_ts(tmem + L::cKV, a + 16, b, idKV, 1);
            mma_bf16_ts(tmem + L::cKV, a, b, idKV, 1);
          }
          mma_commit(&bar[kAFree + buf]);
          if (q == 3) {
            mma_commit(&bar[kKV]);
            mma_commit(&bar[kEmpty + st]);
          }
        }
        __syncwarp();
      }
    }
    if (elect_one()) mma_commit(&bar[kDrainB]);
    __syncwarp();
    mbar_wait(&bar[kDrainB], 0, kWaitNs);
  } else {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      tma_prefetch_desc(&map_k);
      tma_prefetch_desc(&map_v);
      if (OUT) tma_prefetch_desc(&map_q);
    }
    const uint32_t bytes = (uint32_t)((OUT ? 2 : 1) * dkp + dvp) * 256u;
    for (int c = 0; c < n_chunks; ++c) {
      const int st = c & 1;
      if (c >= 2 && !wait(kEmpty + st, (c >> 1) - 1)) break;
      if (lane == 0) {
        const int t0 = t_begin + c * C;
        mbar_arrive_expect_tx(&bar[kFull + st], bytes);
        for (int x = 0; x < dkp; x += 64) {
          if (OUT) tma_load_3d(sm + L::Q + st * kTile + (x >> 6) * kAtom, &map_q, &bar[kFull + st], x, hk, t0);
          tma_load_3d(sm + L::K + st * kTile + (x >> 6) * kAtom, &map_k, &bar[kFull + st], x, hk, t0);
        }
        for (int x = 0; x < dvp; x += 64)
          tma_load_3d(sm + L::V + st * kTile + (x >> 6) * kAtom, &map_v, &bar[kFull + st], x, h, t0);
        *issued = c + 1;
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*dead) {
    // A wait gave up: let the loads in flight land (each wait bounded; the MMAs were drained by their
    // issuing warps), then report.  The results are unspecified.
    if (tid == 0) {
      for (int c = max(0, *issued - 2); c < *issued; ++c) mbar_wait(&bar[kFull + (c & 1)], (uint32_t)((c >> 1) & 1), kWaitNs);
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
  __shared__ int scratch[2 * (kCarryNT / 32) + 8];
  const int h = blockIdx.x % p.h_v, seq = blockIdx.x / p.h_v;
  const Unit un = find_unit<kCarryNT / 32>(p.cu, p.n_seqs, p.total_tokens, p.seg_tokens, -1, seq, scratch);
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
  CUtensorMap mq{}, mk, mv;
  if ((lp.write_O && !make_map_heads(&mq, lp.q, lp.total_tokens, lp.h_k, lp.d_k)) ||
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
  cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay::ALLOC);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(linear_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay::ALLOC);
  if (e != cudaSuccess) return e;
  if (cut || !lp.write_O) {
    linear_tc_kernel<false><<<(unsigned)blocks, NT, Lay::ALLOC, stream>>>(mq, mk, mv, p);
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
    linear_tc_kernel<true><<<(unsigned)blocks, NT, Lay::ALLOC, stream>>>(mq, mk, mv, p);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace gdn
