// C ABI of what the requests of one batch differ by (include/kvr.h): checks of
// arguments, then the launches of k_sample.cu and k_adapt.cu.
#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cstdio>

#include "kvr_batch.cuh"

using namespace kvr;

namespace {

thread_local char g_error[256] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_error, sizeof g_error, fmt, ap);
  va_end(ap);
  return code;
}
int cuda_fail(cudaError_t e, const char* what) { return fail(KVR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e)); }

// SMs and status word of the current device, whose kernels are set up on its first call
constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];
std::atomic<int*> g_status[kMaxDevices];
cudaError_t device_of_call(int* sms, int** status) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices && (*sms = g_sms[dev].load(std::memory_order_acquire)) != 0) {
    *status = g_status[dev].load(std::memory_order_relaxed);   // (stored before)
    return cudaSuccess;
  }
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = sample_setup();
  if (e == cudaSuccess) e = adapt_setup();
  if (e == cudaSuccess) e = adapt_status(status);
  if (e == cudaSuccess && dev < kMaxDevices) {
    g_status[dev].store(*status, std::memory_order_relaxed);
    g_sms[dev].store(*sms, std::memory_order_release);
  }
  return e;
}

constexpr int kMaxSampleRows = 1 << 20;

int type_bytes(int type) { return type == KVR_ACT_F32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool shared_with_any(const Span& out, const Span* in, int n) {
  for (int i = 0; i < n; ++i)
    if (shared(out, in[i])) return true;
  return false;
}

int logits_check(const void* logits, int type, long long stride, int rows, int vocab, const kvr_sampling* s) {
  if (type != KVR_ACT_F32 && type != KVR_ACT_BF16 && type != KVR_ACT_F16)
    return fail(KVR_ERR_ARG, "logits of type %d", type);
  if (rows < 0 || rows > kMaxSampleRows) return fail(KVR_ERR_ARG, "%d rows outside [0, %d]", rows, kMaxSampleRows);
  if (vocab < 1 || vocab > KVR_MAX_VOCAB) return fail(KVR_ERR_ARG, "vocab %d outside [1, %d]", vocab, KVR_MAX_VOCAB);
  if (rows > 1 && stride < vocab) return fail(KVR_ERR_ARG, "the row stride must cover a row");
  if (rows && (!logits || !aligned(logits, type_bytes(type)))) return fail(KVR_ERR_ARG, "missing or misaligned logits");
  if (s && !(aligned(s->temperature, 4) && aligned(s->top_k, 4) && aligned(s->min_p, 4) && aligned(s->top_p, 4)))
    return fail(KVR_ERR_ARG, "misaligned settings");
  return KVR_OK;
}

constexpr int kMaxAdaptRows = 1 << 22;

int run_sample(const SampleParams& p, void* stream) {
  int sms = 0, *status = nullptr;
  cudaError_t e = device_of_call(&sms, &status);
  if (e == cudaSuccess) e = launch_sample(p, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVR_OK : cuda_fail(e, "sample launch");
}

}  // namespace

bool kvr::shared(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.n < 1 || b.n < 1) return false;
  const long long off = (long long)((uintptr_t)b.p - (uintptr_t)a.p);   // of b, from a
  if (off >= a.bytes() || -off >= b.bytes()) return false;
  if (b.n == 1) {
    const long long i = off < a.width ? 0 : (off - a.width) / a.stride + 1;   // the first row that ends behind b's start
    return i < a.n && i * a.stride < off + b.width;
  }
  if (a.n == 1) return shared(b, a);
  if (a.stride != b.stride) return true;
  const long long in = ((off % a.stride) + a.stride) % a.stride;   // of b's rows, from the start of a's
  return in < a.width || in + b.width > a.stride;
}

bool kvr::adapter_site_ok(const kvr_adapter_site* s) {
  if (!s || !s->table || !aligned(s->table, 8) || s->n_adapters < 1 || s->max_rank < 8 || s->max_rank > KVR_MAX_RANK ||
      s->max_rank % 8 || s->k < 8 || s->k % 8 || s->k > 1 << 20 || s->n_parts < 1 || s->n_parts > 3 ||
      (s->type != KVR_ACT_BF16 && s->type != KVR_ACT_F16))
    return false;
  for (int j = 0; j < s->n_parts; ++j)
    if (s->cols[j] < 8 || s->cols[j] % 8 || s->cols[j] > 1 << 20) return false;
  return true;
}

extern "C" {

int kvr_sample(const void* logits, int type, long long stride, int rows, int vocab, const kvr_sampling* settings,
               const float* u, int32_t* token, float* prob, float* dist, long long dist_stride, void* stream) {
  if (int rc = logits_check(logits, type, stride, rows, vocab, settings)) return rc;
  if (rows == 0) return KVR_OK;
  if (!u || !token || !aligned(u, 4) || !aligned(token, 4) || !aligned(prob, 4) || !aligned(dist, 4))
    return fail(KVR_ERR_ARG, "missing or misaligned u, token, prob or dist");
  if (dist && rows > 1 && dist_stride < vocab) return fail(KVR_ERR_ARG, "dist's row stride must cover a row");
  SampleParams p = {};
  if (settings) p.s = *settings;
  const long long n = 4ll * rows, es = type_bytes(type);
  const Span out[3] = {{token, n}, {prob, n}, {dist, rows, rows > 1 ? 4 * dist_stride : 4ll * vocab, 4ll * vocab}};
  const Span in[6] = {{logits, rows, rows > 1 ? es * stride : es * vocab, es * vocab},
                      {u, n}, {p.s.temperature, n}, {p.s.top_k, n}, {p.s.min_p, n}, {p.s.top_p, n}};
  for (int i = 0; i < 3; ++i)
    if (shared_with_any(out[i], in, 6) || shared_with_any(out[i], out, i))
      return fail(KVR_ERR_ARG, "token, prob or dist shares memory with another argument");
  p.logits = logits;
  p.stride = stride;
  p.rows = rows;
  p.vocab = vocab;
  p.type = type;
  p.u = u;
  p.token = token;
  p.prob = prob;
  p.dist = dist;
  p.dist_stride = dist_stride;
  return run_sample(p, stream);
}

size_t kvr_accept_work_bytes(int rows) { return rows < 0 || rows > kMaxSampleRows ? 0 : (size_t)std::max(rows, 1) * 4; }

int kvr_accept(const void* logits, int type, long long stride, int rows, int vocab, const kvr_sampling* settings,
               int n_seq, const int32_t* cu_rows, const int32_t* tokens, const float* draft_probs,
               long long draft_stride, const float* u, const float* u_next, int32_t* accepted, int32_t* next,
               void* work, size_t work_bytes, void* stream) {
  if (int rc = logits_check(logits, type, stride, rows, vocab, settings)) return rc;
  if (n_seq < 1 || n_seq > 65536) return fail(KVR_ERR_ARG, "%d sequences outside [1, 65536]", n_seq);
  if (!cu_rows || !u_next || !accepted || !next || (rows && (!tokens || !u)))
    return fail(KVR_ERR_ARG, "null cu_rows, tokens, u, u_next, accepted or next");
  for (const void* q : {(const void*)cu_rows, (const void*)tokens, (const void*)u, (const void*)u_next,
                        (const void*)accepted, (const void*)next, (const void*)draft_probs})
    if (!aligned(q, 4)) return fail(KVR_ERR_ARG, "misaligned pointer");
  if (draft_probs && rows > 1 && draft_stride < vocab)
    return fail(KVR_ERR_ARG, "the drafts' row stride must cover a row");
  if (!work || !aligned(work, 16) || work_bytes < kvr_accept_work_bytes(rows))
    return fail(KVR_ERR_CAPACITY, "work area missing, misaligned or smaller than %zu bytes", kvr_accept_work_bytes(rows));
  SampleParams p = {};
  if (settings) p.s = *settings;
  const long long n = 4ll * rows, ns = 4ll * n_seq, es = type_bytes(type);
  const Span out[3] = {{accepted, ns}, {next, ns}, {work, n}};
  const Span in[10] = {{logits, rows, rows > 1 ? es * stride : es * vocab, es * vocab},
                       {draft_probs, rows, rows > 1 ? 4 * draft_stride : 4ll * vocab, 4ll * vocab},
                       {rows ? tokens : nullptr, n}, {rows ? u : nullptr, n}, {cu_rows, ns + 4}, {u_next, ns},
                       {p.s.temperature, ns}, {p.s.top_k, ns}, {p.s.min_p, ns}, {p.s.top_p, ns}};
  for (int i = 0; i < 3; ++i)
    if (shared_with_any(out[i], in, 10) || shared_with_any(out[i], out, i))
      return fail(KVR_ERR_ARG, "accepted, next or work shares memory with another argument");
  p.logits = logits;
  p.stride = stride;
  p.rows = rows;
  p.vocab = vocab;
  p.type = type;
  p.u = u;
  p.cu = cu_rows;
  p.n_seq = n_seq;
  p.tokens = tokens;
  p.q = draft_probs;
  p.q_stride = draft_stride;
  p.u_next = u_next;
  p.outcome = static_cast<int32_t*>(work);
  p.accepted = accepted;
  p.next = next;
  return run_sample(p, stream);
}

size_t kvr_adapt_work_bytes(const kvr_adapter_site* site, int rows) {
  if (!adapter_site_ok(site) || rows < 0 || rows > kMaxAdaptRows) return 0;
  return adapt_work_bytes(*site, std::max(rows, 1));
}

int kvr_adapt(const kvr_adapter_site* site, const void* x, long long x_stride, const int32_t* cu_rows,
              const int32_t* which, int n_seq, int rows, const void* base, long long base_stride, void* out,
              long long out_stride, int out_type, void* work, size_t work_bytes, void* stream) {
  if (!adapter_site_ok(site))
    return fail(KVR_ERR_ARG, "a site's table, adapters, ranks, widths or type are out of their range");
  if (rows < 0 || rows > kMaxAdaptRows) return fail(KVR_ERR_ARG, "%d rows outside [0, %d]", rows, kMaxAdaptRows);
  if (n_seq < 1 || n_seq > kAdaptMaxSeqs) return fail(KVR_ERR_ARG, "%d sequences outside [1, %d]", n_seq, kAdaptMaxSeqs);
  if (out_type != site->type && out_type != KVR_ACT_F32) return fail(KVR_ERR_ARG, "outputs of type %d", out_type);
  if (rows == 0) return KVR_OK;
  if (!x || !cu_rows || !which || !out) return fail(KVR_ERR_ARG, "null x, cu_rows, which or out");
  if (!aligned(x, 16) || !aligned(base, 16) || !aligned(out, 16) || !aligned(cu_rows, 4) || !aligned(which, 4))
    return fail(KVR_ERR_ARG, "x, base and out must be 16-byte aligned");
  long long n = 0;
  for (int j = 0; j < site->n_parts; ++j) n += site->cols[j];
  if (rows == 1) x_stride = site->k, base_stride = out_stride = n;   // (one row's stride means nothing)
  if (x_stride < site->k || x_stride % 8 || out_stride < n || out_stride % 8 ||
      (base && (base_stride < n || base_stride % 8)))
    return fail(KVR_ERR_ARG, "row strides must cover a row and be multiples of 8");
  if (base == out && base_stride != out_stride) return fail(KVR_ERR_ARG, "base is out, but its stride is another");
  if (!work || !aligned(work, 16) || work_bytes < adapt_work_bytes(*site, rows))
    return fail(KVR_ERR_CAPACITY, "work area missing, misaligned or smaller than %zu bytes", adapt_work_bytes(*site, rows));
  const long long size = out_type == KVR_ACT_F32 ? 4 : 2;
  const Span to[2] = {{out, rows, size * out_stride, size * n}, {work, (long long)adapt_work_bytes(*site, rows)}};
  const Span in[5] = {{x, rows, 2 * x_stride, 2ll * site->k},
                      {base == out ? nullptr : base, rows, size * base_stride, size * n},
                      {cu_rows, 4ll * n_seq + 4}, {which, 4ll * n_seq},
                      {site->table, (long long)sizeof(kvr_adapter) * site->n_adapters}};
  if (shared_with_any(to[0], in, 5) || shared_with_any(to[1], in, 5) || shared(to[0], to[1]))
    return fail(KVR_ERR_ARG, "out or work shares memory with another argument");
  AdaptParams p = {};
  p.site = *site;
  p.x = x;
  p.x_stride = x_stride;
  p.cu = cu_rows;
  p.which = which;
  p.n_seq = n_seq;
  p.rows = rows;
  p.base = base;
  p.base_stride = base_stride;
  p.out = out;
  p.out_stride = out_stride;
  p.out_type = out_type;
  p.part = static_cast<float*>(work);
  int sms = 0;
  cudaError_t e = device_of_call(&sms, &p.status);
  if (e == cudaSuccess) e = launch_adapt(p, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVR_OK : cuda_fail(e, "adapt launch");
}

int kvr_batch_sync(void* stream) {
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int sms = 0, word = 0, *status = nullptr;
  cudaError_t e = device_of_call(&sms, &status);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&word, status, sizeof word, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && word) {
    e = cudaMemsetAsync(status, 0, sizeof word, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess) return fail(KVR_ERR_TIMEOUT, "a wait in a kernel of kvr_adapt gave up");
  }
  return e == cudaSuccess ? KVR_OK : cuda_fail(e, "status readback");
}

int kvr_batch_selftest_wait(void* stream) {
  int sms = 0, *status = nullptr;
  cudaError_t e = device_of_call(&sms, &status);
  if (e == cudaSuccess) e = launch_wait_probe(status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVR_OK : cuda_fail(e, "wait probe launch");
}

const char* kvr_batch_error(void) { return g_error; }

}  // extern "C"
