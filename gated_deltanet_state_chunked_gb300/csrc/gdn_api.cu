// C ABI of libgdn.so: argument checks, dispatch to the kernels, status word.
#include <cuda_runtime.h>

#include <cstdio>
#include <cstring>
#include <cstdarg>
#include <mutex>
#include <string>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

thread_local std::string g_last_error;
thread_local void* g_stage_event = nullptr;  // cudaEvent_t to record between prep and scan, once
constexpr unsigned long long kDefaultWaitNs = 2000000000ull;
thread_local unsigned long long g_wait_ns = kDefaultWaitNs;  // next compose call's wait limit, once

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

__device__ int g_status;  // sticky per-device status (one copy per device that loads the library)

constexpr int kMaxGridY = 65535;    // v-heads of one launch of the prompt and decode kernels
constexpr int kMaxRows = INT32_MAX - 1023;  // tokens or drafts of a serving call: the kernels step past the last in 32 bits
constexpr int kMaxVocab = 1 << 19;  // sums of 2^-44 fixed-point probabilities are at most 2^63

int check_head_dims(const gdn_dims* d) {
  if (d->h_k <= 0 || d->h_v <= 0) return fail(GDN_ERR_ARG, "h_k and h_v must be positive");
  if (d->h_v % d->h_k != 0) return fail(GDN_ERR_SHAPE, "h_v (%d) must be a multiple of h_k (%d)", d->h_v, d->h_k);
  if (d->d_k <= 0 || d->d_v <= 0 || d->d_k > kMaxHead || d->d_v > kMaxHead || d->d_k % 8 || d->d_v % 8)
    return fail(GDN_ERR_UNSUPPORTED, "d_k=%d, d_v=%d: need multiples of 8 in [8, %d]", d->d_k, d->d_v, kMaxHead);
  return GDN_OK;
}

int check_token_dims(const gdn_dims* d) {
  if (d->n_seqs < 0 || d->total_tokens < 0) return fail(GDN_ERR_ARG, "negative n_seqs or total_tokens");
  if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return fail(GDN_ERR_UNSUPPORTED, "dtype %d", d->dtype);
  if (d->flags & ~(GDN_QK_L2NORM | GDN_STATE_ONLY | GDN_PRECISE | GDN_SCALAR_DECAY))
    return fail(GDN_ERR_ARG, "unknown flag bits 0x%x", d->flags);
  return check_head_dims(d);
}

// Stream-ordered scratch: one private memory pool per device that keeps its memory
// (release threshold = max), so after the first call allocations are pool hits.
int scratch_pool(cudaMemPool_t* out) {
  static std::mutex mu;
  static cudaMemPool_t pools[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= 64) return fail(GDN_ERR_UNSUPPORTED, "device ordinal %d", dev);
  std::lock_guard<std::mutex> lock(mu);
  if (!pools[dev]) {
    cudaMemPoolProps props = {};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = dev;
    e = cudaMemPoolCreate(&pools[dev], &props);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemPoolCreate");
    uint64_t keep = UINT64_MAX;
    e = cudaMemPoolSetAttribute(pools[dev], cudaMemPoolAttrReleaseThreshold, &keep);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemPoolSetAttribute");
  }
  *out = pools[dev];
  return GDN_OK;
}

}  // namespace

// Argument checks of gdn_replay and gdn_replay_noalloc (one set of rules for both): fills *p,
// sets *nothing_to_do for an empty batch.
int check_replay_args(const gdn_dims* dims, const void* q, const void* k, const void* v, const float* g,
                      const float* beta, const int32_t* cu_seqlens, const float* S0, void* O_out, float* S_out,
                      SimtParams* p, bool* nothing_to_do) {
  g_last_error.clear();
  *nothing_to_do = false;
  if (!dims) return fail(GDN_ERR_ARG, "dims is NULL");
  int rc = check_token_dims(dims);
  if (rc) return rc;
  const bool state_only = dims->flags & GDN_STATE_ONLY;
  if (dims->n_seqs == 0) {
    *nothing_to_do = true;
    return GDN_OK;
  }
  if (!cu_seqlens || !S_out) return fail(GDN_ERR_ARG, "cu_seqlens and S_out are required");
  if (!state_only && !O_out) return fail(GDN_ERR_ARG, "O_out is NULL without GDN_STATE_ONLY");
  if (dims->total_tokens > 0 && (!q || !k || !v || !g || !beta))
    return fail(GDN_ERR_ARG, "q, k, v, g and beta are required when total_tokens > 0");
  const void* p16[] = {q, k, v, O_out, S0, S_out};
  for (const void* ptr : p16)
    if (ptr && !aligned(ptr, 16)) return fail(GDN_ERR_ALIGN, "q, k, v, O, S0 and S_out must be 16-byte aligned");
  if (!aligned(g, 4) || !aligned(beta, 4) || !aligned(cu_seqlens, 4))
    return fail(GDN_ERR_ALIGN, "g, beta and cu_seqlens must be 4-byte aligned");
  int* status = device_status_word();
  if (!status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  *p = SimtParams{};
  p->q = q; p->k = k; p->v = v; p->g = g; p->beta = beta; p->cu = cu_seqlens; p->S0 = S0;
  p->O = state_only ? nullptr : O_out;
  p->S_out = S_out; p->T_out = nullptr;
  p->n_seqs = dims->n_seqs; p->total_tokens = dims->total_tokens;
  p->h_k = dims->h_k; p->h_v = dims->h_v; p->d_k = dims->d_k; p->d_v = dims->d_v;
  p->augmented = 0; p->l2norm = (dims->flags & GDN_QK_L2NORM) ? 1 : 0;
  p->write_O = state_only ? 0 : 1; p->scale = dims->scale; p->status = status;
  p->scalar_decay = (dims->flags & GDN_SCALAR_DECAY) ? 1 : 0;
  return GDN_OK;
}

int report_error(int code, const char* message) { return fail(code, "%s", message); }

void* take_stage_event() {
  void* e = g_stage_event;
  g_stage_event = nullptr;
  return e;
}

unsigned long long take_wait_limit_ns() {
  const unsigned long long ns = g_wait_ns;
  g_wait_ns = kDefaultWaitNs;
  return ns;
}

int* device_status_word() {  // (looked up in each call: the address is the current context's)
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess) return nullptr;
  return static_cast<int*>(p);
}

}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_abi_version(void) { return GDN_ABI_VERSION; }

void gdn_set_stage_event(void* event) { g_stage_event = event; }

void gdn_set_wait_limit_ns(uint64_t ns) { g_wait_ns = ns; }

const char* gdn_last_error(void) { return g_last_error.c_str(); }

size_t gdn_workspace_bytes(const gdn_dims* dims) {
  if (!dims || dims->total_tokens <= 0 || dims->n_seqs <= 0 || dims->h_v <= 0) return 0;
  if (dims->dtype == GDN_BF16 && !(dims->flags & GDN_PRECISE) && dims->d_k == kMaxHead && dims->d_v == kMaxHead)
    return replay_tc_workspace_bytes(dims->n_seqs, dims->total_tokens, dims->h_v);
  return simt_records_bytes(dims->n_seqs, dims->total_tokens, dims->h_v);  // fp32 path: its records
}

int gdn_replay(const gdn_dims* dims, const void* q, const void* k, const void* v, const float* g,
               const float* beta, const int32_t* cu_seqlens, const float* S0, void* O_out, float* S_out,
               void* stream) {
  SimtParams p;
  bool nothing = false;
  const int rc = check_replay_args(dims, q, k, v, g, beta, cu_seqlens, S0, O_out, S_out, &p, &nothing);
  if (rc || nothing) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dims->dtype == GDN_BF16 && !(dims->flags & GDN_PRECISE) && replay_tc_supported(p)) {
    const size_t bytes = replay_tc_workspace_bytes(p.n_seqs, p.total_tokens, p.h_v);
    cudaMemPool_t pool = nullptr;
    int prc = scratch_pool(&pool);
    if (prc) return prc;
    void* ws = nullptr;
    cudaError_t e = cudaMallocFromPoolAsync(&ws, bytes, pool, st);
    if (e != cudaSuccess) return fail(GDN_ERR_NOMEM, "scratch of %zu bytes: %s", bytes, cudaGetErrorString(e));
    e = launch_replay_tc(p, ws, bytes, st);
    const cudaError_t ef = cudaFreeAsync(ws, st);
    if (e != cudaSuccess) return cuda_fail(e, "gdn_replay tensor-core launch");
    if (ef != cudaSuccess) return cuda_fail(ef, "scratch release");
    return GDN_OK;
  }
  // fp32 path in two passes: the chunk-shared quantities (norms, gates, (I + A)^{-1}, P) once per
  // (chunk, v-head) into pool scratch, then the row slices of each state read them.
  const size_t bytes = simt_records_bytes(p.n_seqs, p.total_tokens, p.h_v);
  cudaMemPool_t pool = nullptr;
  int prc = scratch_pool(&pool);
  if (prc) return prc;
  void* ws = nullptr;
  cudaError_t e = cudaMallocFromPoolAsync(&ws, bytes, pool, st);
  if (e != cudaSuccess) return fail(GDN_ERR_NOMEM, "scratch of %zu bytes: %s", bytes, cudaGetErrorString(e));
  e = launch_replay_simt_two_pass(p, dims->dtype == GDN_BF16, ws, bytes, st);
  const cudaError_t ef = cudaFreeAsync(ws, st);
  if (e != cudaSuccess) return cuda_fail(e, "gdn_replay launch");
  if (ef != cudaSuccess) return cuda_fail(ef, "scratch release");
  return GDN_OK;
}

int gdn_chunk_operator(const gdn_dims* dims, const void* k, const float* g, const float* beta, const void* v,
                       const int32_t* cu_seqlens, float* T_out, float* Slocal_out, void* stream) {
  g_last_error.clear();
  if (!dims) return fail(GDN_ERR_ARG, "dims is NULL");
  int rc = check_token_dims(dims);
  if (rc) return rc;
  if (dims->n_seqs == 0) return GDN_OK;
  if (!cu_seqlens && dims->n_seqs != 1) return fail(GDN_ERR_ARG, "cu_seqlens may be NULL only for one chunk");
  if (!T_out || !Slocal_out) return fail(GDN_ERR_ARG, "T_out and Slocal_out are required");
  if (dims->total_tokens > 0 && (!k || !v || !g || !beta))
    return fail(GDN_ERR_ARG, "k, v, g and beta are required when total_tokens > 0");
  const void* p16[] = {k, v, T_out, Slocal_out};
  for (const void* p : p16)
    if (p && !aligned(p, 16)) return fail(GDN_ERR_ALIGN, "k, v, T_out and Slocal_out must be 16-byte aligned");
  if (!aligned(g, 4) || !aligned(beta, 4) || !aligned(cu_seqlens, 4))
    return fail(GDN_ERR_ALIGN, "g, beta and cu_seqlens must be 4-byte aligned");
  int* status = device_status_word();
  if (!status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");

  SimtParams p{};
  p.q = nullptr; p.k = k; p.v = v; p.g = g; p.beta = beta; p.cu = cu_seqlens; p.S0 = nullptr;
  p.O = nullptr; p.S_out = Slocal_out; p.T_out = T_out;
  p.n_seqs = dims->n_seqs; p.total_tokens = dims->total_tokens;
  p.h_k = dims->h_k; p.h_v = dims->h_v; p.d_k = dims->d_k; p.d_v = dims->d_v;
  p.augmented = 1; p.l2norm = (dims->flags & GDN_QK_L2NORM) ? 1 : 0;
  p.write_O = 0; p.scale = 1.f; p.status = status;
  p.scalar_decay = (dims->flags & GDN_SCALAR_DECAY) ? 1 : 0;
  // Two passes: the chunk-shared quantities once per (chunk, v-head) into pool scratch, then the
  // row slices of the augmented state [S; P] read them.
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t bytes = simt_records_bytes(p.n_seqs, p.total_tokens, p.h_v);
  cudaMemPool_t pool = nullptr;
  int prc = scratch_pool(&pool);
  if (prc) return prc;
  void* ws = nullptr;
  cudaError_t e = cudaMallocFromPoolAsync(&ws, bytes, pool, st);
  if (e != cudaSuccess) return fail(GDN_ERR_NOMEM, "scratch of %zu bytes: %s", bytes, cudaGetErrorString(e));
  e = launch_replay_simt_two_pass(p, dims->dtype == GDN_BF16, ws, bytes, st);
  const cudaError_t ef = cudaFreeAsync(ws, st);
  if (e != cudaSuccess) return cuda_fail(e, "gdn_chunk_operator launch");
  if (ef != cudaSuccess) return cuda_fail(ef, "scratch release");
  return GDN_OK;
}

int gdn_compose(const gdn_dims* dims, int32_t K, const float* const* T, const float* const* Slocal,
                const float* S_in, float* S_out, void* stream) {
  g_last_error.clear();
  if (!dims) return fail(GDN_ERR_ARG, "dims is NULL");
  int rc = check_head_dims(dims);
  if (rc) return rc;
  if (K < 0 || K > kMaxCompose) return fail(GDN_ERR_ARG, "K=%d outside [0, %d]", K, kMaxCompose);
  if (!S_out) return fail(GDN_ERR_ARG, "S_out is required");
  if (K > 0 && (!T || !Slocal)) return fail(GDN_ERR_ARG, "T and Slocal arrays are required when K > 0");
  ComposeParams p{};
  for (int j = 0; j < K; ++j) {
    if (!T[j] || !Slocal[j]) return fail(GDN_ERR_ARG, "T[%d] or Slocal[%d] is NULL", j, j);
    if (!aligned(T[j], 16) || !aligned(Slocal[j], 16)) return fail(GDN_ERR_ALIGN, "T[%d]/Slocal[%d] not 16-byte aligned", j, j);
    if (T[j] == S_out || Slocal[j] == S_out) return fail(GDN_ERR_ARG, "S_out aliases an input");
    p.T[j] = T[j];
    p.Slocal[j] = Slocal[j];
  }
  if ((S_in && !aligned(S_in, 16)) || !aligned(S_out, 16)) return fail(GDN_ERR_ALIGN, "S_in/S_out not 16-byte aligned");
  if (S_in && S_in == S_out) return fail(GDN_ERR_ARG, "S_out aliases S_in");
  p.S_in = S_in; p.S_out = S_out; p.K = K; p.h = dims->h_v; p.d_k = dims->d_k; p.d_v = dims->d_v;
  p.status = device_status_word();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  p.wait_ns = take_wait_limit_ns();
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = compose_tc_supported(p) ? launch_compose_tc(p, st) : launch_compose_simt(p, st);
  if (e != cudaSuccess) return cuda_fail(e, "gdn_compose launch");
  return GDN_OK;
}

int gdn_linear_attn(const gdn_dims* dims, const void* q, const void* k, const void* v, const float* log_decay,
                    const int32_t* cu_seqlens, const float* S0, void* O_out, float* S_out, void* stream) {
  g_last_error.clear();
  if (!dims) return fail(GDN_ERR_ARG, "dims is NULL");
  if (dims->flags & ~GDN_STATE_ONLY) return fail(GDN_ERR_ARG, "gdn_linear_attn takes GDN_STATE_ONLY only, got 0x%x", dims->flags);
  int rc = check_token_dims(dims);
  if (rc) return rc;
  if (dims->h_v > kMaxGridY) return fail(GDN_ERR_UNSUPPORTED, "h_v=%d above %d", dims->h_v, kMaxGridY);
  if (dims->total_tokens > kMaxRows) return fail(GDN_ERR_UNSUPPORTED, "total_tokens=%d above %d", dims->total_tokens, kMaxRows);
  // (a launch has a block for each segment, of 64 tokens or more unless it is a sequence's last, and v-head)
  if (((long long)dims->n_seqs + dims->total_tokens / 64) * dims->h_v > INT32_MAX)
    return fail(GDN_ERR_UNSUPPORTED, "n_seqs=%d, total_tokens=%d, h_v=%d: too many pieces of work", dims->n_seqs,
                dims->total_tokens, dims->h_v);
  const bool state_only = dims->flags & GDN_STATE_ONLY;
  if (dims->n_seqs == 0) return GDN_OK;
  if (!cu_seqlens || !S_out || !log_decay) return fail(GDN_ERR_ARG, "cu_seqlens, log_decay and S_out are required");
  if (!state_only && !O_out && dims->total_tokens > 0) return fail(GDN_ERR_ARG, "O_out is NULL without GDN_STATE_ONLY");
  if (dims->total_tokens > 0 && ((!q && !state_only) || !k || !v))
    return fail(GDN_ERR_ARG, "q (unless GDN_STATE_ONLY), k and v are required when total_tokens > 0");
  const void* p16[] = {q, k, v, O_out, S0, S_out};
  for (const void* ptr : p16)
    if (ptr && !aligned(ptr, 16)) return fail(GDN_ERR_ALIGN, "q, k, v, O, S0 and S_out must be 16-byte aligned");
  if (!aligned(log_decay, 4) || !aligned(cu_seqlens, 4))
    return fail(GDN_ERR_ALIGN, "log_decay and cu_seqlens must be 4-byte aligned");
  LinearParams p{};
  p.q = q; p.k = k; p.v = v; p.log_decay = log_decay; p.cu = cu_seqlens; p.S0 = S0;
  p.O = state_only ? nullptr : O_out; p.S_out = S_out;
  p.n_seqs = dims->n_seqs; p.total_tokens = dims->total_tokens;
  p.h_k = dims->h_k; p.h_v = dims->h_v; p.d_k = dims->d_k; p.d_v = dims->d_v;
  p.write_O = state_only ? 0 : 1; p.scale = dims->scale;
  p.status = device_status_word();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  size_t bytes = 0;
  void* ws = nullptr;
  cudaError_t e = linear_workspace_bytes(p, dims->dtype == GDN_BF16, &bytes), ef = cudaSuccess;
  if (e != cudaSuccess) return cuda_fail(e, "gdn_linear_attn set-up");
  if (bytes) {
    cudaMemPool_t pool = nullptr;
    rc = scratch_pool(&pool);
    if (rc) return rc;
    e = cudaMallocFromPoolAsync(&ws, bytes, pool, st);
    if (e != cudaSuccess) return fail(GDN_ERR_NOMEM, "scratch of %zu bytes: %s", bytes, cudaGetErrorString(e));
  }
  e = launch_linear(p, dims->dtype == GDN_BF16, ws, st);
  if (ws) ef = cudaFreeAsync(ws, st);
  if (e != cudaSuccess) return cuda_fail(e, "gdn_linear_attn launch");
  if (ef != cudaSuccess) return cuda_fail(ef, "scratch release");
  return GDN_OK;
}

int gdn_decode(const gdn_dims* dims, int32_t n_slots, const void* q, const void* k, const void* v, const float* g,
               const float* beta, const int32_t* slots, const int32_t* counts, float* S_pool, void* O_out,
               void* stream) {
  g_last_error.clear();
  if (!dims) return fail(GDN_ERR_ARG, "dims is NULL");
  gdn_dims base = *dims;
  base.flags &= ~(GDN_HEAD_DECAY | GDN_KEEP_STATE);
  int rc = check_token_dims(&base);
  if (rc) return rc;
  const uint32_t fl = dims->flags;
  const bool state_only = fl & GDN_STATE_ONLY, keep = fl & GDN_KEEP_STATE, head = fl & GDN_HEAD_DECAY;
  if (fl & GDN_PRECISE) return fail(GDN_ERR_ARG, "gdn_decode takes no GDN_PRECISE (every sum is in fp32)");
  if (state_only && keep) return fail(GDN_ERR_ARG, "GDN_STATE_ONLY with GDN_KEEP_STATE leaves nothing to do");
  if (head && (fl & GDN_SCALAR_DECAY)) return fail(GDN_ERR_ARG, "GDN_HEAD_DECAY and GDN_SCALAR_DECAY exclude each other");
  if (dims->h_v > kMaxGridY) return fail(GDN_ERR_UNSUPPORTED, "h_v=%d above %d", dims->h_v, kMaxGridY);
  if (dims->total_tokens > kMaxRows) return fail(GDN_ERR_UNSUPPORTED, "total_tokens=%d above %d", dims->total_tokens, kMaxRows);
  if (n_slots < 0) return fail(GDN_ERR_ARG, "negative n_slots");
  if (dims->n_seqs == 0 || dims->total_tokens == 0) return GDN_OK;
  if (dims->total_tokens % dims->n_seqs)
    return fail(GDN_ERR_SHAPE, "total_tokens (%d) must be n_seqs (%d) windows of one length", dims->total_tokens, dims->n_seqs);
  if (!slots && dims->n_seqs > n_slots)
    return fail(GDN_ERR_SHAPE, "%d requests on %d slots without a slot list", dims->n_seqs, n_slots);
  if (!S_pool && n_slots > 0) return fail(GDN_ERR_ARG, "S_pool is required");
  if (!k || !v || !g || (!q && !state_only)) return fail(GDN_ERR_ARG, "q (unless GDN_STATE_ONLY), k, v and g are required");
  if (head ? beta != nullptr : beta == nullptr)
    return fail(GDN_ERR_ARG, "beta is required, and must be NULL with GDN_HEAD_DECAY");
  if (!state_only && !O_out) return fail(GDN_ERR_ARG, "O_out is NULL without GDN_STATE_ONLY");
  const void* p16[] = {q, k, v, O_out, S_pool};
  for (const void* ptr : p16)
    if (ptr && !aligned(ptr, 16)) return fail(GDN_ERR_ALIGN, "q, k, v, O and S_pool must be 16-byte aligned");
  if (!aligned(g, 4) || !aligned(beta, 4) || !aligned(slots, 4) || !aligned(counts, 4))
    return fail(GDN_ERR_ALIGN, "g, beta, slots and counts must be 4-byte aligned");
  DecodeParams p{};
  p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta; p.slots = slots; p.counts = counts; p.S = S_pool;
  p.O = state_only ? nullptr : O_out;
  p.n = dims->n_seqs; p.window = dims->total_tokens / dims->n_seqs; p.n_slots = n_slots;
  p.h_k = dims->h_k; p.h_v = dims->h_v; p.d_k = dims->d_k; p.d_v = dims->d_v;
  p.v_per_k = p.h_v / p.h_k;
  p.family = head ? kHeadDecay : (fl & GDN_SCALAR_DECAY) ? kScalarDecay : kDelta;
  p.l2norm = (fl & GDN_QK_L2NORM) ? 1 : 0; p.state_only = state_only ? 1 : 0; p.keep = keep ? 1 : 0;
  p.scale = dims->scale;
  p.status = device_status_word();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  const cudaError_t e = launch_decode(p, dims->dtype == GDN_BF16, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_decode launch");
  return GDN_OK;
}

int gdn_verify_draft(const gdn_verify_dims* dims, const void* target, const void* draft, const int32_t* drafted,
                     const int32_t* draft_lens, const float* uniforms, int32_t* counts_out, int32_t* tokens_out,
                     void* stream) {
  g_last_error.clear();
  if (!dims) return fail(GDN_ERR_ARG, "dims is NULL");
  if (dims->n_seqs < 0 || dims->n_draft < 0) return fail(GDN_ERR_ARG, "negative n_seqs or n_draft");
  if (dims->vocab <= 0) return fail(GDN_ERR_ARG, "vocab must be positive");
  if (dims->dtype != GDN_F32 && dims->dtype != GDN_BF16) return fail(GDN_ERR_UNSUPPORTED, "dtype %d", dims->dtype);
  if (dims->n_draft > kMaxRows) return fail(GDN_ERR_UNSUPPORTED, "n_draft=%d above %d", dims->n_draft, kMaxRows);
  if (dims->vocab > kMaxVocab) return fail(GDN_ERR_UNSUPPORTED, "vocab=%d above %d", dims->vocab, kMaxVocab);
  if (dims->target_stride < dims->vocab || (draft && dims->draft_stride < dims->vocab))
    return fail(GDN_ERR_SHAPE, "a row stride is below vocab (%d)", dims->vocab);
  if (dims->n_seqs == 0) return GDN_OK;
  if (!target || !uniforms || !counts_out || !tokens_out)
    return fail(GDN_ERR_ARG, "target, uniforms, counts_out and tokens_out are required");
  if (dims->n_draft > 0 && !drafted) return fail(GDN_ERR_ARG, "drafted is required when n_draft > 0");
  const size_t es = dims->dtype == GDN_BF16 ? 2 : 4;
  if (!aligned(target, es) || !aligned(draft, es)) return fail(GDN_ERR_ALIGN, "target and draft must be aligned to their type");
  if (!aligned(drafted, 4) || !aligned(draft_lens, 4) || !aligned(uniforms, 4) || !aligned(counts_out, 4) || !aligned(tokens_out, 4))
    return fail(GDN_ERR_ALIGN, "drafted, draft_lens, uniforms, counts_out and tokens_out must be 4-byte aligned");
  VerifyParams p{};
  p.target = target; p.draft = dims->n_draft > 0 ? draft : nullptr; p.drafted = drafted; p.draft_lens = draft_lens;
  p.uniforms = uniforms; p.counts = counts_out; p.tokens = tokens_out;
  p.target_stride = dims->target_stride; p.draft_stride = dims->draft_stride;
  p.n = dims->n_seqs; p.n_draft = dims->n_draft; p.vocab = dims->vocab;
  p.status = device_status_word();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  const cudaError_t e = launch_verify(p, dims->dtype == GDN_BF16, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_verify_draft launch");
  return GDN_OK;
}

int gdn_get_status(void* stream) {
  g_last_error.clear();
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "stream");
  int st = 0;
  e = cudaMemcpyFromSymbol(&st, g_status, sizeof(int));
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  if (st != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e, "status clear");
    return fail(st, "device reported status %d", st);
  }
  return GDN_OK;
}

}  // extern "C"
