// Work division and shared pieces of gdn_paged_attn's kernels.
//
// An item is one (request, key head, row tile): the query rows of up to `tile_tokens` consecutive new
// tokens, all the query heads of the key head, against the keys that any of them sees, in units of BN keys
// (an item that sees no key is one unit).  The items of a call, request after request, head after head, form one line of
// units, COST places ahead of each one's for what an item costs besides (its queries, the filling and draining of the
// pipeline, its outputs), and each of G CTAs takes an equal stretch of the line, whatever the lengths are: lengths are
// read on the device, so that no host code could deal the items out, and a long request next to short ones fills the
// GPU.  (Without those places a CTA that met eleven short items took 147 us where the others took 119: 64 tokens over
// up to 6,000 keys.)  An item that several CTAs share leaves partial results (normalised rows, running maximum and
// sum) in scratch, which paged_join_kernel puts together in the order of the keys: results do not depend on timing.
#pragma once

#include <climits>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "gdn_internal.cuh"
#include "umma.cuh"

namespace gdn {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A request: its rows of q, its new tokens (0: nothing to do), its tokens in the cache.
struct Request {
  int q0, len, kv;
};

// Partial results: what CTA c does of an item that an earlier CTA began lies in slot 2 c, its part of one that it
// begins and does not finish in slot 2 c + 1.
struct Shared {
  int req, head, tile, last;  // an item that CTA c began and CTA `last` finished; req < 0: none
  Request r;
  int pad;
};
struct Scratch {
  float* rows;   // [2 G][BM][d]
  float2* stat;  // [2 G][BM] (maximum in log2 units, sum)
  Shared* shared;  // [G]
};
inline size_t scratch_bytes(int G, int BM, int d) {
  return (size_t)2 * G * BM * (d * sizeof(float) + sizeof(float2)) + (size_t)G * sizeof(Shared);
}
inline Scratch scratch_at(void* ws, int G, int BM, int d) {
  Scratch s;
  s.rows = static_cast<float*>(ws);
  s.stat = reinterpret_cast<float2*>(s.rows + (size_t)2 * G * BM * d);
  s.shared = reinterpret_cast<Shared*>(s.stat + (size_t)2 * G * BM);
  return s;
}

// `top`: the largest of the offsets before request i (a range that starts below it is malformed).
__device__ __forceinline__ Request request_of(const PagedParams& p, int i, int top, bool* bad) {
  Request r;
  int b;
  if (p.cu) {
    r.q0 = p.cu[i];
    b = p.cu[i + 1];
  } else {
    const int w = p.total / p.n;
    r.q0 = i * w;
    b = r.q0 + w;
  }
  r.kv = p.kv_lens[i];
  const bool range = r.q0 >= 0 && r.q0 >= top && b >= r.q0 && b <= p.total && b - r.q0 <= p.max_q;
  *bad = !range || (r.kv >= 0 && (unsigned)r.kv > ((unsigned)p.width << p.page_shift));
  r.len = *bad || r.kv < 0 ? 0 : b - r.q0;
  return r;
}
__device__ __forceinline__ int top_of(const PagedParams& p, int i) { return p.cu ? max(p.cu[i], p.cu[i + 1]) : INT_MIN; }

// The first key that position `pos` sees.
__device__ __forceinline__ int low_of(const PagedParams& p, int pos) {
  return p.window && pos >= p.window ? pos - p.window + 1 : 0;
}

// Keys that the tokens [t0, t0 + n) of a request see: [lo, hi).
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span span_of(const PagedParams& p, const Request& r, int t0, int n) {
  const int base = r.kv - r.len;  // position of the first new token
  Span s;
  s.hi = max(0, min(r.kv, base + min(t0 + n, r.len)));
  s.lo = low_of(p, base + t0);
  return s;
}
template <int BN>
__device__ __forceinline__ int units_of(const Span& s) {
  return s.hi > s.lo ? (s.hi + BN - 1) / BN - s.lo / BN : 1;
}

// Walks the stretch of one CTA.  All threads hold the same values.
template <int BN, int COST>
struct Walk {
  int req, top;    // request, and the largest offset before it
  Request r;
  int head, tile;  // the item
  Span span;
  int units, at;   // the item's units, and the next of them
  int left;        // places of the stretch from that unit on (units may be left of it while it is above 0)
  long long begin; // the item's first place
  long long total;
  int G;

  __device__ __forceinline__ void set_tile(const PagedParams& p, int tile_tokens) {
    span = span_of(p, r, tile * tile_tokens, tile_tokens);
    units = units_of<BN>(span);
  }
  // Units taken from the item in this step; the CTA works on units [at, at + n).
  __device__ __forceinline__ int step() const { return min(units - at, left); }
  __device__ __forceinline__ void advance(const PagedParams& p, int tile_tokens, int n) {
    left -= n;
    at += n;
    if (at < units) return;  // (the stretch ends inside the item)
    left -= COST;
    if (left <= 0) return;
    begin += COST + units;
    at = 0;
    if ((tile + 1) * tile_tokens < r.len) {
      ++tile;
    } else {
      tile = 0;
      if (++head == p.h_kv) {
        head = 0;
        do {
          top = max(top, top_of(p, req));
          ++req;
          bool bad;
          r = request_of(p, req, top, &bad);
        } while (r.len == 0);
      }
    }
    set_tile(p, tile_tokens);
  }
  // The CTA that works on the item's last unit.
  __device__ __forceinline__ int last_cta() const { return (int)(((begin + COST + units) * G - 1) / total); }
};

struct PlanSmem {
  long long sum[32];
  int top[32];
  long long start, per_head;
  int req, top_before;
};

// Places of one key head's items of this lane's request.  Long chunks (more than 32 tiles) by the whole warp.
template <int BN, int COST>
__device__ __forceinline__ long long places_of(const PagedParams& p, const Request& r, int tile_tokens) {
  constexpr int kAlone = 32;
  long long n = 0;
  if (r.len <= kAlone * tile_tokens)
    for (int t = 0; t < r.len; t += tile_tokens) n += COST + units_of<BN>(span_of(p, r, t, tile_tokens));
  for (unsigned many = __ballot_sync(0xffffffffu, r.len > kAlone * tile_tokens); many; many &= many - 1) {
    const int l = __ffs(many) - 1, lane = threadIdx.x & 31;
    const Request x = {__shfl_sync(0xffffffffu, r.q0, l), __shfl_sync(0xffffffffu, r.len, l), __shfl_sync(0xffffffffu, r.kv, l)};
    const int tiles = (x.len - 1) / tile_tokens + 1;
    long long sum = 0;
    for (int t = lane; t < tiles; t += 32) sum += COST + units_of<BN>(span_of(p, x, t * tile_tokens, tile_tokens));
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == l) n = sum;
  }
  return n;
}

// Finds this CTA's stretch: false if it has none.  All NT threads of the CTA call it; CTA 0 reports
// malformed requests.
template <int BN, int COST, int NT>
__device__ bool plan(const PagedParams& p, int tile_tokens, PlanSmem& sm, Walk<BN, COST>& w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long total = 0, u0 = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long sum = 0;
    int top = INT_MIN;
    for (int first = 0; first < p.n; first += NT) {
      const int i = first + tid;
      int incl_top = i < p.n ? top_of(p, i) : INT_MIN;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl_top, o);
        if (lane >= o) incl_top = max(incl_top, x);
      }
      int before = __shfl_up_sync(0xffffffffu, incl_top, 1);
      if (lane == 0) before = INT_MIN;
      if (lane == 31) sm.top[warp] = incl_top;
      __syncthreads();
      before = max(before, top);
      for (int x = 0; x < NT / 32; ++x) {
        if (x < warp) before = max(before, sm.top[x]);
        top = max(top, sm.top[x]);
      }
      Request r = {0, 0, -1};
      if (i < p.n) {
        bool bad;
        r = request_of(p, i, before, &bad);
        if (bad && pass == 0 && blockIdx.x == 0) atomicExch(p.status, GDN_ERR_SHAPE);
      }
      const long long per_head = places_of<BN, COST>(p, r, tile_tokens), mine = per_head * p.h_kv;
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) sm.sum[warp] = incl;
      __syncthreads();
      long long start = sum + incl - mine;
      for (int x = 0; x < NT / 32; ++x) {
        if (x < warp) start += sm.sum[x];
        sum += sm.sum[x];
      }
      if (pass == 0 && p.n <= NT) {  // (one round: nothing needs to be read again)
        total = sum;
        const int G = (int)min((long long)gridDim.x, total);
        u0 = G ? total * blockIdx.x / G : 0;
      }
      if ((pass == 1 || p.n <= NT) && mine > 0 && start <= u0 && u0 < start + mine) {
        sm.start = start;
        sm.per_head = per_head;
        sm.req = i;
        sm.top_before = before;
      }
      __syncthreads();
    }
    if (p.n <= NT) break;
    if (pass == 0) {
      total = sum;
      const int G = (int)min((long long)gridDim.x, total);
      u0 = G ? total * blockIdx.x / G : 0;
    }
  }
  w.total = total;
  w.G = (int)min((long long)gridDim.x, total);
  if ((int)blockIdx.x >= w.G) return false;
  const long long end = total * (blockIdx.x + 1) / w.G;
  w.req = sm.req;
  w.top = sm.top_before;
  bool bad;
  w.r = request_of(p, w.req, w.top, &bad);
  long long u = u0 - sm.start;
  w.head = (int)(u / sm.per_head);
  u -= w.head * sm.per_head;
  for (int first = 0;; first += 32) {  // the tile that place u lies in, 32 of them at a time
    const int t = first + lane;
    const int mine = t * (long long)tile_tokens < w.r.len ? COST + units_of<BN>(span_of(p, w.r, t * tile_tokens, tile_tokens)) : 0;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned there = __ballot_sync(0xffffffffu, u < incl);
    if (there) {
      const int l = __ffs(there) - 1;
      w.tile = first + l;
      u -= __shfl_sync(0xffffffffu, incl - mine, l);
      break;
    }
    u -= __shfl_sync(0xffffffffu, incl, 31);
  }
  w.set_tile(p, tile_tokens);
  w.begin = u0 - u;
  w.at = max(0, (int)u - COST);
  w.left = (int)(end - (w.begin + COST + w.at));  // (a stretch has fewer places than 2^31 units)
  return w.left > 0;
}

// Where a row's key j lies: element offset in the pages, or -1 for a page outside the cache (reported).
__device__ __forceinline__ int page_of(const PagedParams& p, int req, int j) {
  const int page = p.table[req * p.table_stride + (j >> p.page_shift)];
  if ((unsigned)page >= (unsigned)p.n_pages) {
    atomicExch(p.status, GDN_ERR_SHAPE);
    return -1;
  }
  return page;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ void store_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

// 16 bytes of a row of the pages or of q, as fp32 numbers.
__device__ __forceinline__ void load16(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// One row by itself, over the keys [lo, hi) that it sees, for rows whose output a tile leaves infinite or NaN
// though their sum of weights is a number: an infinite or NaN value at a key that the row does not see, but
// its tile does, has done that (0 * inf), or an unnormalised sum past fp32, or a value that the row does see.  The
// maximum and sum first, then the sum of values with weights that add up to 1.  One warp; lane l returns values l, l + 32, ...
template <typename T>
__device__ __noinline__ void row_again(const PagedParams& p, int req, int head, int h, int row, int lo, int hi, float (&o)[4],
                                       float* m_out, float* l_out) {
  constexpr int VEC = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  const T* q = static_cast<const T*>(p.q) + (int64_t)row * p.q_stride + (int64_t)h * p.d;
  const T* kp = static_cast<const T*>(p.k) + head * p.k_head;
  const T* vp = static_cast<const T*>(p.v) + head * p.v_head;
  const int mask = (1 << p.page_shift) - 1;
  const float s2 = p.scale * kLog2e;
  auto score = [&](int j, int* page) {
    *page = j < hi ? page_of(p, req, j) : -1;
    if (*page < 0) return -CUDART_INF_F;
    const T* k = kp + *page * p.k_page + (int64_t)(j & mask) * p.k_token;
    float s = 0.f;
    for (int x = 0; x < p.d; x += VEC) {
      float a[VEC], b[VEC];
      load16(q + x, a);
      load16(k + x, b);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s = fmaf(a[i], b[i], s);
    }
    return s * s2;
  };
  float m = -CUDART_INF_F, l = 0.f;
  for (int j0 = lo; j0 < hi; j0 += 32) {  // (a lane's own maximum and sum)
    int page;
    const float s = score(j0 + lane, &page), m_new = fmaxf(m, s), ref = m_new == -CUDART_INF_F ? 0.f : m_new;
    l = l * exp2f(m - ref) + (page >= 0 ? exp2f(s - ref) : 0.f);
    m = m_new;
  }
  float top = m;
  for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  const float ref = top == -CUDART_INF_F ? 0.f : top;
  l *= exp2f(m - ref);
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float f = 1.f / l;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = 0.f;
  for (int j0 = lo; j0 < hi; j0 += 32) {
    int page;
    const float s = score(j0 + lane, &page), e = exp2f(s - ref) * f;
    for (int x = 0; x < min(32, hi - j0); ++x) {
      const float w = __shfl_sync(0xffffffffu, e, x);
      const int pg = __shfl_sync(0xffffffffu, page, x);
      if (pg < 0) continue;
      const T* v = vp + pg * p.v_page + (int64_t)((j0 + x) & mask) * p.v_token;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < p.d) o[i] = fmaf(w, to_f(v[lane + 32 * i]), o[i]);
    }
  }
  *m_out = top;
  *l_out = l;
}
// Whether a row with such an output is worth it (l: its sum of weights): with a NaN or infinite score every value is
// NaN already, as with no weight at all.
__device__ __forceinline__ bool worth_again(float l) { return l > 0.f && l <= 3.402823466e38f; }

// Row r of a tile of item (head, tile): its token of the request and its query head.
struct Row {
  int t, h;
  bool live;
};
__device__ __forceinline__ Row row_of(const PagedParams& p, const Request& rq, int head, int tile, int tile_tokens, int r) {
  Row x;
  const int tt = r / p.group;
  x.t = tile * tile_tokens + tt;
  x.h = head * p.group + (r - tt * p.group);
  x.live = tt < tile_tokens && x.t < rq.len;
  return x;
}
// Normalisation of a finished row: the factor of its sums.  A row that sees no key is zero; one whose keys
// all score -inf is NaN, as its softmax is.
__device__ __forceinline__ float row_factor(float l, bool sees) { return sees ? 1.f / l : 0.f; }
__device__ __forceinline__ float row_lse(float m, float l, bool sees) {
  return sees ? (l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2) : -CUDART_INF_F;
}

// row_again for a row of a piece (keys [first, end) of the item's), and its results to where the piece's go.
template <typename T>
__device__ __forceinline__ void redo_row(const PagedParams& p, const Scratch& s, const Request& rq, int req, int head,
                                         const Row& x, int first, int end, bool whole, size_t slot_row) {
  const int lane = threadIdx.x & 31, pos = rq.kv - rq.len + x.t;
  const int lo = max(first, low_of(p, pos)), hi = min(end, pos + 1);
  float o[4], m, l;
  row_again<T>(p, req, head, x.h, rq.q0 + x.t, lo, hi, o, &m, &l);
  const size_t out = (size_t)(rq.q0 + x.t) * p.h_q + x.h;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = lane + 32 * i;
    if (c >= p.d) continue;
    if (!whole) s.rows[slot_row * p.d + c] = l == 0.f ? 0.f : o[i];
    else store_f(static_cast<T*>(p.O) + out * p.d + c, o[i]);
  }
  if (lane == 0) {
    if (!whole) s.stat[slot_row] = float2{m, l};
    else if (p.lse) p.lse[out] = row_lse(m, l, pos >= 0);
  }
}

// Puts the partial results of shared items together.
cudaError_t launch_join(const PagedParams& p, int bf16, const Scratch& s, int G, int BM, int tile_tokens, cudaStream_t stream);
cudaError_t launch_simt(const PagedParams& p, int bf16, void* workspace, cudaStream_t stream);
cudaError_t simt_workspace(const PagedParams& p, int bf16, size_t* bytes);
cudaError_t launch_tc(const PagedParams& p, void* workspace, cudaStream_t stream);
bool tc_supported(const PagedParams& p);
cudaError_t launch_split(const PagedParams& p, void* workspace, cudaStream_t stream);
cudaError_t split_workspace(const PagedParams& p, size_t* bytes);
cudaError_t tc_workspace(const PagedParams& p, size_t* bytes);

inline cudaError_t sm_count(int* n) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace paged
}  // namespace gdn
