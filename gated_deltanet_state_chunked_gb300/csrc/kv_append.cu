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

// cos and sin of angle = position * inv_freq.  The product of a 31-bit position and a 24-bit frequency and its
// remainder by 2 pi are taken in fp64 (in fp32 a product near 10^5 is off by 4e-3 already); what is left is
// within [-pi, pi], where fp32 sine and cosine are exact to their last bits.
__device__ __forceinline__ float2 turn_of(int position, float inv_freq) {
  const double a = (double)position * (double)inv_freq;
  const double r = fma(-rint(a * 0.15915494309189535), 6.283185307179586, a);
  float2 t;
  sincosf((float)r, &t.y, &t.x);
  return t;
}

// A 16-byte piece of a row: VEC values of type T, as fp32 numbers.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int VEC = 4;
  static __device__ __forceinline__ void get(const float* p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  static __device__ __forceinline__ void put(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = float4{x[0], x[1], x[2], x[3]};
  }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ void get(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    *reinterpret_cast<uint4*>(p) = uint4{u[0], u[1], u[2], u[3]};
  }
};

// A token's rows: h_q queries, h_kv keys, h_kv values.
template <typename T>
struct Rows {
  const T* q;
  const T* k;
  const T* v;
  T* q_out;
  T* k_out;  // null: the token has no place
  T* v_out;
};
template <typename T>
__device__ __forceinline__ bool row_at(const PagedParams& p, const Rows<T>& rows, int i, const T** src, T** dst) {
  const int n_q = rows.q ? p.h_q : 0;
  if (i < n_q) {
    *src = rows.q + (int64_t)i * p.d;
    *dst = rows.q_out + (int64_t)i * p.d;
    return true;
  }
  const int h = i - n_q;
  const bool key = h < p.h_kv;
  const int hh = key ? h : h - p.h_kv;
  *src = (key ? rows.k : rows.v) + (int64_t)hh * p.d;
  *dst = key ? rows.k_out : rows.v_out;
  if (*dst) *dst += key ? hh * p.k_head : hh * p.v_head;
  return key;
}

// One CTA a token.  Its request is found by all threads at once; the turns of its pairs are computed once
// for all heads.  Bound by HBM where there are many tokens, by the chain request -> page and angles -> rows where
// there are few.  SPLIT: pairs lie half a rotation apart (else side by side); VECTOR: a rotated part of whole
// 16-byte pieces (else pair by pair).
template <typename T, bool SPLIT, bool VECTOR>
__global__ void __launch_bounds__(kAppendNT) kv_append_kernel(PagedParams p) {
  constexpr int VEC = Piece<T>::VEC;
  __shared__ float2 turn[kMaxHead / 2];
  __shared__ int found;
  const int tid = threadIdx.x, t = blockIdx.x;
  const int half = p.rotary / 2;
  // the request that holds the token: the first whose range does (a malformed one is reported by the first CTA)
  if (tid == 0) found = INT_MAX;
  __syncthreads();
  int req = 0;
  if (p.cu) {
    for (int i = tid; i < p.n; i += kAppendNT)
      if (p.cu[i] <= t && t < p.cu[i + 1]) atomicMin(&found, i);
    __syncthreads();
    req = found;
  } else {
    req = t / (p.total / p.n);
  }
  bool skip = req == INT_MAX, bad = false;
  Request r = {0, 0, -1};
  if (!skip) {
    int above = 0;
    if (p.cu) {
      const int start = p.cu[req];
      for (int i = tid; i < req; i += kAppendNT) above |= p.cu[i] > start;
      above = __syncthreads_or(above);
    }
    r = request_of(p, req, above ? INT_MAX : INT_MIN, &bad);
    skip = r.len == 0;
  }
  if (blockIdx.x == 0) {
    // (an offset above a later one is found between neighbours or with the largest one before)
    int top = INT_MIN, wrong = 0;
    if (tid < 32)
      for (int first = 0; first < p.n; first += 32) {
        const int i = first + tid;
        int incl = i < p.n ? top_of(p, i) : INT_MIN;
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, incl, o);
          if (tid >= o) incl = max(incl, x);
        }
        int before = __shfl_up_sync(0xffffffffu, incl, 1);
        before = max(top, tid ? before : INT_MIN);
        if (i < p.n) {
          bool b;
          request_of(p, i, before, &b);
          wrong |= b;
        }
        top = max(top, __shfl_sync(0xffffffffu, incl, 31));
      }
    if (wrong) atomicExch(p.status, GDN_ERR_SHAPE);
  }
  if (skip) return;
  const int pos = r.kv - r.len + (t - r.q0);
  if (tid < half) {
    int axis = 0;
    for (int pairs = 0; axis + 1 < p.n_axes; ++axis) {
      pairs += p.sections[axis];
      if (tid < pairs) break;
    }
    turn[tid] = turn_of(p.positions ? p.positions[(int64_t)axis * p.total + t] : pos, p.inv_freq[tid]);
  }
  Rows<T> rows;
  rows.q = p.q ? static_cast<const T*>(p.q) + t * p.q_stride : nullptr;
  rows.q_out = static_cast<T*>(p.O) + (int64_t)t * p.h_q * p.d;
  rows.k = static_cast<const T*>(p.k) + t * p.k_stride;
  rows.v = static_cast<const T*>(p.v) + t * p.v_stride;
  rows.k_out = rows.v_out = nullptr;
  if (pos >= 0) {
    const int page = p.table[req * p.table_stride + (pos >> p.page_shift)];
    if ((unsigned)page < (unsigned)p.n_pages) {
      const int64_t slot = pos & ((1 << p.page_shift) - 1);
      rows.k_out = static_cast<T*>(p.k_pages) + page * p.k_page + slot * p.k_token;
      rows.v_out = static_cast<T*>(p.v_pages) + page * p.v_page + slot * p.v_token;
    } else if (tid == 0) {
      atomicExch(p.status, GDN_ERR_SHAPE);
    }
  }
  __syncthreads();
  const int n_rows = (p.q ? p.h_q : 0) + 2 * p.h_kv;
  if (VECTOR) {
    // (where pairs lie apart, a rotated row's pieces are done two at once and those of its second half passed over)
    const int turned = SPLIT ? half / VEC : p.rotary / VEC, pieces = p.d / VEC;
    for (int i = tid; i < n_rows * pieces; i += kAppendNT) {
      const int row = i / pieces, c = i - row * pieces;
      const T* src;
      T* dst;
      const bool rotate = row_at(p, rows, row, &src, &dst);
      if (!dst) continue;
      float a[VEC];
      if (!rotate || c * VEC >= p.rotary) {
        Piece<T>::get(src + c * VEC, a);
        Piece<T>::put(dst + c * VEC, a);
      } else if (SPLIT) {
        if (c >= turned) continue;
        float b[VEC], x[VEC], y[VEC];
        Piece<T>::get(src + c * VEC, a);
        Piece<T>::get(src + half + c * VEC, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float2 w = turn[c * VEC + j];
          x[j] = a[j] * w.x - b[j] * w.y;
          y[j] = b[j] * w.x + a[j] * w.y;
        }
        Piece<T>::put(dst + c * VEC, x);
        Piece<T>::put(dst + half + c * VEC, y);
      } else {
        Piece<T>::get(src + c * VEC, a);
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const float2 w = turn[(c * VEC + j) / 2];
          const float x = a[j] * w.x - a[j + 1] * w.y, y = a[j + 1] * w.x + a[j] * w.y;
          a[j] = x;
          a[j + 1] = y;
        }
        Piece<T>::put(dst + c * VEC, a);
      }
    }
  } else {
    for (int i = tid; i < n_rows * (p.d / 2); i += kAppendNT) {
      const int row = i / (p.d / 2), c = i - row * (p.d / 2);
      const T* src;
      T* dst;
      const bool rotate = row_at(p, rows, row, &src, &dst);
      if (!dst) continue;
      const bool turned = rotate && c < half;
      const int i0 = SPLIT && c < half ? c : 2 * c, i1 = SPLIT && c < half ? c + half : 2 * c + 1;
      const float a = to_f(src[i0]), b = to_f(src[i1]);
      const float2 w = turned ? turn[c] : float2{1.f, 0.f};
      store_f(dst + i0, turned ? a * w.x - b * w.y : a);
      store_f(dst + i1, turned ? b * w.x + a * w.y : b);
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
