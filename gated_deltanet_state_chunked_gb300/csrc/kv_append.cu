// gdn_kv_append: new keys and values into a paged cache, keys and queries rotated by their positions.
#include "paged_work.cuh"

namespace gdn {
namespace {

using paged::Request;
using paged::request_of;
using paged::store_f;
using paged::to_f;
using paged::top_of;

constexpr int kAppendNT = 128;

// cos and sin of the angle position * inv_freq.  In revolutions, as whole multiples of 2^-64, what counts of the product is
// what is left of it modulo 2^64: one integer multiplication, exact but for the frequency's own last bit (2^-64 of a
// revolution, 2^-33 at a position of 2^31).  (In fp32 a product near 10^5 is off by 4e-3 already; reducing it in
// fp64, at the rate of this GPU's fp64, kept the other warps waiting: 8,192 tokens in 49 us.)
__device__ __forceinline__ uint64_t step_of(float inv_freq) {  // inv_freq / (2 pi) in 2^-64, modulo 2^64
  const uint32_t u = __float_as_uint(inv_freq);
  const int e = (int)(u >> 23 & 255);
  const uint64_t m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);  // |inv_freq| = m 2^(max(e, 1) - 150)
  constexpr uint64_t kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;  // 2^64 / (2 pi) and its fraction
  const uint64_t low = m * kHigh + __umul64hi(m, kLow), high = __umul64hi(m, kHigh) + (low < m * kHigh);
  const int down = 150 - max(e, 1);  // (at least 0: below 2^24, see turn_of)
  const uint64_t g = down == 0 ? low : down < 64 ? low >> down | high << (64 - down) : down < 128 ? high >> (down - 64) : 0ull;
  return u >> 31 ? 0ull - g : g;
}
__device__ __forceinline__ float2 turn_of(int position, float inv_freq) {
  float2 t;
  if (fabsf(inv_freq) < 16777216.f) {
    const uint64_t x = (uint64_t)(int64_t)position * step_of(inv_freq);
    sincospif((float)(int32_t)(x >> 32) * 0x1p-31f, &t.y, &t.x);
  } else {  // (no frequency that positions are told apart by, or no number)
    double s, c;
    sincos((double)position * (double)inv_freq, &s, &c);
    t = float2{(float)c, (float)s};
  }
  return t;
}

// A 16-byte piece of a row: VEC values of type T, as fp32 numbers and back.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int VEC = 4;
  static __device__ __forceinline__ void open(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 close(const float (&x)[4]) {
    return uint4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
  }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ void open(const uint4& v, float (&x)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 close(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    return uint4{u[0], u[1], u[2], u[3]};
  }
};

// A token's rows, from and to: h_q queries (if any), then h_kv keys, then h_kv values.
template <typename T>
struct Rows {
  const T *q, *k, *v;
  T *q_to, *k_to, *v_to;  // (k_to null: the token has no place)
  __device__ __forceinline__ const T* from(const PagedParams& p, int n_q, int i) const {
    return i < n_q ? q + i * p.d : i < n_q + p.h_kv ? k + (i - n_q) * p.d : v + (i - n_q - p.h_kv) * p.d;
  }
  __device__ __forceinline__ T* to(const PagedParams& p, int n_q, int i) const {
    return i < n_q ? q_to + i * p.d : !k_to ? nullptr : i < n_q + p.h_kv ? k_to + (i - n_q) * p.k_head : v_to + (i - n_q - p.h_kv) * p.v_head;
  }
};

// Two fp32 operations in one instruction (values as register pairs).
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The request that holds token t: the first whose range does (its number; -1: none, or a malformed one).  One warp.
__device__ __forceinline__ int find_request(const PagedParams& p, int t, Request* r) {
  const int lane = threadIdx.x & 31;
  *r = Request{0, 0, -1};
  if (!p.cu) {
    const int w = p.total / p.n, i = t / w;
    *r = Request{i * w, w, p.kv_lens[i]};
    return i;
  }
  for (int first = 0; first < p.n; first += 128) {
    int begin[4], end[4], kv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = first + 32 * j + lane;
      const bool there = i < p.n;
      begin[j] = there ? p.cu[i] : INT_MAX;
      end[j] = there ? p.cu[i + 1] : INT_MAX;
      kv[j] = there ? p.kv_lens[i] : -1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned holds = __ballot_sync(0xffffffffu, begin[j] <= t && t < end[j]);
      if (holds) {
        const int l = __ffs(holds) - 1, req = first + 32 * j + l;
        r->q0 = __shfl_sync(0xffffffffu, begin[j], l);
        r->len = __shfl_sync(0xffffffffu, end[j], l) - r->q0;
        r->kv = __shfl_sync(0xffffffffu, kv[j], l);
        int above = 0;  // (an earlier offset above the range's first: a malformed range)
        for (int i = lane; i < req; i += 32) above |= p.cu[i] > r->q0;
        const bool bad = __any_sync(0xffffffffu, above) || r->q0 < 0 || r->q0 + r->len > p.total || r->len > p.max_q;
        return bad ? -1 : req;
      }
    }
  }
  return -1;
}

// One CTA a token.  Its rows are read ahead of what they do not depend on: its request (found by one warp), its page, and
// the turns of its pairs, which are computed once for all heads; a thread turns the same pairs of several rows.  Bound by HBM
// where there are many tokens, by the chain request -> page -> rows out where there are few.  Measured: 8,192 tokens of 48 rows
// of 128 bf16 values 43 us, 4.7 TB/s (about 750 instructions a warp beside the copies); one token 3.5 us in a graph.  SPLIT: pairs lie half a rotation
// apart (else side by side); VECTOR: a rotated part of whole 16-byte pieces (else pair by pair).
template <typename T, bool SPLIT, bool VECTOR>
__global__ void __launch_bounds__(kAppendNT, 6) kv_append_kernel(PagedParams p) {
  constexpr int VEC = Piece<T>::VEC, kAhead = 3;
  __shared__ __align__(16) float cosine[kMaxHead / 2], sine[kMaxHead / 2];
  __shared__ int found;
  __shared__ Request request;
  const int tid = threadIdx.x, t = blockIdx.x;
  const int half = p.rotary / 2, n_q = p.q ? p.h_q : 0, turned_rows = n_q + p.h_kv;
  Rows<T> rows;
  rows.q = static_cast<const T*>(p.q) + t * p.q_stride;
  rows.k = static_cast<const T*>(p.k) + t * p.k_stride;
  rows.v = static_cast<const T*>(p.v) + t * p.v_stride;
  rows.q_to = static_cast<T*>(p.O) + (int64_t)t * p.h_q * p.d;
  rows.k_to = rows.v_to = nullptr;
  // Queries and keys: `per_row` threads to a row, each with piece `at` of rows row0, row0 + step, ...  Where pairs lie apart,
  // the rotated pieces are done two at once, at and at + apart, and then come the row's last pieces.
  const int pieces = p.d / VEC, apart = SPLIT ? half / VEC : 0, per_row = pieces - apart;
  const int row0 = tid / per_row, step = kAppendNT / per_row, c = tid - row0 * per_row;
  const bool mine = row0 < step, turns = c * VEC < (SPLIT ? half : p.rotary);
  const int at = turns ? c : c + apart;
  // Values: piece v_at of rows v_row0, v_row0 + v_step, ...
  const int v_row0 = tid / pieces, v_step = kAppendNT / pieces, v_at = tid - v_row0 * pieces;
  const bool v_mine = v_row0 < v_step;
  uint4 a[kAhead], b[kAhead], v[kAhead];
  auto read = [&](int first) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int row = first + row0 + k * step;
      if (mine && row < turned_rows) {
        const T* src = rows.from(p, n_q, row);
        a[k] = *reinterpret_cast<const uint4*>(src + at * VEC);
        if (SPLIT && turns) b[k] = *reinterpret_cast<const uint4*>(src + half + at * VEC);
      }
    }
  };
  auto read_values = [&](int first) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int row = first + v_row0 + k * v_step;
      if (v_mine && row < p.h_kv) v[k] = *reinterpret_cast<const uint4*>(rows.v + row * p.d + v_at * VEC);
    }
  };
  if (VECTOR) {
    read(0);
    read_values(0);
  }
  const float inv_freq = tid < half ? p.inv_freq[tid] : 0.f;
  if (tid < 32) {
    Request x;
    const int req = find_request(p, t, &x);
    if (tid == 0) {
      found = req;
      request = x;
    }
    if (blockIdx.x == 0) {  // what is malformed is reported by the first CTA
      int top = INT_MIN, wrong = 0;
      for (int first = 0; first < p.n; first += 32) {
        const int i = first + tid;
        int incl = i < p.n ? top_of(p, i) : INT_MIN;
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (tid >= o) incl = max(incl, y);
        }
        int before = __shfl_up_sync(0xffffffffu, incl, 1);
        before = max(top, tid ? before : INT_MIN);
        if (i < p.n) {
          bool bad;
          request_of(p, i, before, &bad);
          wrong |= bad;
        }
        top = max(top, __shfl_sync(0xffffffffu, incl, 31));
      }
      if (wrong) atomicExch(p.status, GDN_ERR_SHAPE);
    }
  }
  __syncthreads();
  const int req = found;
  const Request r = request;
  if (req < 0 || r.kv < 0 || (unsigned)r.kv > ((unsigned)p.width << p.page_shift)) return;
  const int pos = r.kv - r.len + (t - r.q0);
  if (tid < half) {
    int axis = 0;
    for (int pairs = 0; axis + 1 < p.n_axes; ++axis) {
      pairs += p.sections[axis];
      if (tid < pairs) break;
    }
    const float2 w = turn_of(p.positions ? p.positions[(int64_t)axis * p.total + t] : pos, inv_freq);
    cosine[tid] = w.x;
    sine[tid] = w.y;
  }
  if (pos >= 0) {
    const int page = p.table[req * p.table_stride + (pos >> p.page_shift)];
    if ((unsigned)page < (unsigned)p.n_pages) {
      const int64_t slot = pos & ((1 << p.page_shift) - 1);
      rows.k_to = static_cast<T*>(p.k_pages) + page * p.k_page + slot * p.k_token;
      rows.v_to = static_cast<T*>(p.v_pages) + page * p.v_page + slot * p.v_token;
    } else if (tid == 0) {
      atomicExch(p.status, GDN_ERR_SHAPE);
    }
  }
  __syncthreads();
  if (VECTOR) {
    // the turns of this thread's pairs: VEC of them where they lie apart, VEC / 2 side by side
    constexpr int W = SPLIT ? VEC : VEC / 2;
    float wc[W], ws[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
      wc[e] = turns ? cosine[c * W + e] : 1.f;
      ws[e] = turns ? sine[c * W + e] : 0.f;
    }
    for (int first = 0; first < turned_rows; first += kAhead * step) {
      if (first > 0) read(first);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int row = first + row0 + k * step;
        if (!mine || row >= turned_rows) continue;
        T* dst = rows.to(p, n_q, row);
        if (!dst) continue;
        if (turns) {
          float x[VEC], y[VEC];
          Piece<T>::open(a[k], x);
          if (SPLIT) {
            Piece<T>::open(b[k], y);
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
              const uint64_t xx = pair(x[e], x[e + 1]), yy = pair(y[e], y[e + 1]), cc = pair(wc[e], wc[e + 1]);
              unpair(fma2(yy, pair(-ws[e], -ws[e + 1]), mul2(xx, cc)), x[e], x[e + 1]);
              unpair(fma2(xx, pair(ws[e], ws[e + 1]), mul2(yy, cc)), y[e], y[e + 1]);
            }
            *reinterpret_cast<uint4*>(dst + half + at * VEC) = Piece<T>::close(y);
          } else {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
              const float z = x[e] * wc[e / 2] - x[e + 1] * ws[e / 2];
              x[e + 1] = x[e + 1] * wc[e / 2] + x[e] * ws[e / 2];
              x[e] = z;
            }
          }
          a[k] = Piece<T>::close(x);
        }
        *reinterpret_cast<uint4*>(dst + at * VEC) = a[k];
      }
    }
    if (!rows.v_to) return;
    for (int first = 0; first < p.h_kv; first += kAhead * v_step) {
      if (first > 0) read_values(first);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int row = first + v_row0 + k * v_step;
        if (v_mine && row < p.h_kv) *reinterpret_cast<uint4*>(rows.v_to + row * p.v_head + v_at * VEC) = v[k];
      }
    }
  } else {
    const int n_rows = turned_rows + p.h_kv;
    for (int i = tid; i < n_rows * (p.d / 2); i += kAppendNT) {
      const int row = i / (p.d / 2), cc = i - row * (p.d / 2);
      const T* src = rows.from(p, n_q, row);
      T* dst = rows.to(p, n_q, row);
      if (!dst) continue;
      const bool turned = row < turned_rows && cc < half;
      const int i0 = SPLIT && cc < half ? cc : 2 * cc, i1 = SPLIT && cc < half ? cc + half : 2 * cc + 1;
      const float x = to_f(src[i0]), y = to_f(src[i1]);
      store_f(dst + i0, turned ? x * cosine[cc] - y * sine[cc] : x);
      store_f(dst + i1, turned ? y * cosine[cc] + x * sine[cc] : y);
    }
  }
}

template <typename T>
cudaError_t launch(const PagedParams& p, cudaStream_t stream) {
  constexpr int VEC = Piece<T>::VEC;
  const bool split = !p.neighbours, vector = (split ? p.rotary / 2 : p.rotary) % VEC == 0;
  if (split && vector) kv_append_kernel<T, true, true><<<p.total, kAppendNT, 0, stream>>>(p);
  else if (split) kv_append_kernel<T, true, false><<<p.total, kAppendNT, 0, stream>>>(p);
  else if (vector) kv_append_kernel<T, false, true><<<p.total, kAppendNT, 0, stream>>>(p);
  else kv_append_kernel<T, false, false><<<p.total, kAppendNT, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const PagedParams& p, int bf16, cudaStream_t stream) {
  return bf16 ? launch<__nv_bfloat16>(p, stream) : launch<float>(p, stream);
}

}  // namespace gdn
