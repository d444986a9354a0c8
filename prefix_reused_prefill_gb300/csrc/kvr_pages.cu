// C ABI of the paged 4-bit cache (include/kvr.h): checks, the work area's
// layout, and which kernels a call launches.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>

#include "kvr_pages.cuh"

using namespace kvr;

struct kvr_pages {
  kvr_pages_config cfg;
  PagesDev dev;
  PageAttend attend;      // the work buffers of the attention
  PageAttendTc attend_tc;
  int device = 0;
  int ctas = 0;           // one per SM
  int rows = 0, max_add = 0, n_seq = 0;   // of the last plan
  size_t layer_bytes = 0;
  char err[256] = "";
};

namespace {

constexpr size_t kAlign = 256;
// Rows of a sequence and KV head (rows * group) up to which the split kernel
// takes the sequence: 64 where every sequence of the step has so few, but 16 where
// the tensor-memory kernel runs anyway.  Four conversations over 15k tokens take, by
// this and by that kernel: of 4 rows in groups of 7, 35 and 52 us, of 8 in groups of 4,
// 57 and 74, of 8 in groups of 7, 52 and 52; of 16 in groups of 4, 102 and 74, where
// the split kernel costs more but takes the keys of bf16 rows unrounded.  12 conversations
// of 1 to 120 rows, group 4, over up to 4k tokens: 31 us, 37 with 32; large batches lean
// the other way: 64 of 7 to 70 rows, group 7, over up to 16k 274 us, 258 with 32.
constexpr int kPageMany = 64, kPageManyBeside = 16;
// Pages (of one KV head and 8 rows) per CTA up to which the split kernel takes all
// the step's rows: it needs one launch and about 12 us, the tensor-memory kernel
// two and 22, but a page costs it 450 cycles for each 8 rows.  126 rows (group 7)
// over 1024 / 8192 / 16000 / 32000 tokens, 7 to 213 pages a CTA: 12.6 / 24.3 / 36.1 /
// 59.0 us, by the tensor-memory kernel 22.5 / 29.5 / 34.7 / 39.7.  (The host
// knows how long the sequences can be, not how long they are.)
constexpr int kPageFew = 100;
// key blocks a CTA of the tensor-memory kernel takes at least: 254 rows over
// 1668 tokens take 35.4 us with 2, 36.2 with 3 and 38.1 with 5, where fewer CTAs
// run longer but leave fewer parts to merge; 18 rows over 2048: 23.7, 24.7, 27.3
constexpr int kPageMinUnits = 2;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool valid(const kvr_pages_config* c) {
  if (!c) return false;
  const int mx = 1 << 22;
  return c->n_pages >= 1 && c->n_pages <= (1 << 24) && c->n_layers >= 1 && c->n_layers <= 1024 &&
         c->n_kv_heads >= 1 && c->n_kv_heads <= 1024 && c->n_q_heads >= c->n_kv_heads &&
         c->n_q_heads % c->n_kv_heads == 0 && c->n_q_heads / c->n_kv_heads <= 64 &&
         // unit counts of the attention stay below 2^31
         (long long)c->n_pages * c->n_kv_heads <= (1ll << 26) && (c->head_dim == 64 || c->head_dim == 128) &&
         c->max_seqs >= 1 && c->max_seqs <= kPageMaxSeqs && c->max_len >= 1 && c->max_len <= mx &&
         c->max_rows >= 1 && c->max_rows <= mx && (c->act == KVR_ACT_BF16 || c->act == KVR_ACT_F16) &&
         c->rope_theta > 0.f && c->norm_eps >= 0.f && std::isfinite(c->rope_theta) && std::isfinite(c->norm_eps);
}

struct Layout {
  size_t status, info, count, counters, lens, cu, free_list, row_seq, row_pos, row_slot, table, rope, rope_rest, ml,
      part, ml_tc, part_tc, shared, total;
  int width;
};
Layout layout(const kvr_pages_config* c) {
  Layout L;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = align_up(at + bytes);
    return o;
  };
  L.width = (c->max_len + kPage - 1) / kPage;
  // zeroed by kvr_pages_create, in one piece: status .. cu
  L.status = take(8);
  L.info = take(8);
  L.counters = take(kPageAttnMaxCtas * 4);
  L.lens = take((size_t)c->max_seqs * 4);
  L.cu = take((size_t)(c->max_seqs + 1) * 4);
  L.count = take(4);
  L.free_list = take((size_t)c->n_pages * 4);
  L.row_seq = take((size_t)c->max_rows * 4);
  L.row_pos = take((size_t)c->max_rows * 4);
  L.row_slot = take((size_t)c->max_rows * 4);
  L.table = take((size_t)c->max_seqs * L.width * 4);
  L.rope = take((size_t)c->max_len * (c->head_dim / 2) * sizeof(float2));
  L.rope_rest = take((size_t)c->max_len * (c->head_dim / 2) * sizeof(__half2));
  L.ml = take((size_t)kPageAttnPartRows * sizeof(float2));
  L.part = take((size_t)kPageAttnPartRows * c->head_dim * sizeof(float));
  L.ml_tc = take((size_t)kPageTcPartRows * sizeof(float2));
  L.part_tc = take((size_t)kPageTcPartRows * c->head_dim * sizeof(float));
  L.shared = take((size_t)kPageAttnMaxCtas * sizeof(PageShared));
  L.total = at;
  return L;
}

int fail(kvr_pages* c, int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(c->err, sizeof c->err, fmt, ap);
  va_end(ap);
  return code;
}
int cuda_fail(kvr_pages* c, cudaError_t e, const char* what) {
  return fail(c, KVR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// the handle's device for the length of a call
struct OnDevice {
  int before = -1;
  explicit OnDevice(int device) {
    int now = device;
    if (cudaGetDevice(&now) == cudaSuccess && now != device && cudaSetDevice(device) == cudaSuccess) before = now;
  }
  ~OnDevice() {
    if (before >= 0) cudaSetDevice(before);
  }
};

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// checks that append, read and attend share; the kernels' view of the layer
int layer_call(kvr_pages* c, int layer, int rows, PagesDev* dev) {
  if (layer < 0 || layer >= c->cfg.n_layers) return fail(c, KVR_ERR_ARG, "bad layer %d", layer);
  if (rows != c->rows) return fail(c, KVR_ERR_ARG, "%d rows, but the plan has %d", rows, c->rows);
  *dev = c->dev;
  dev->layer_off = (long long)(c->layer_bytes * layer);
  return KVR_OK;
}

// Do n rows of w bytes, s bytes apart from a on, share a byte with the len bytes from b on?
bool overlap(const void* a, long long s, long long n, long long w, const void* b, long long len) {
  const long long off = (long long)((uintptr_t)b - (uintptr_t)a);   // of b, from a
  // the first row that ends behind b's start
  const long long i = off < w ? 0 : (off - w) / s + 1;
  return i < n && i * s < off + len;
}

bool stride_ok(long long stride, long long row) { return stride >= row && stride % 8 == 0 && stride < (1ll << 40); }

}  // namespace

const kvr_pages_config& kvr::pages_config(const kvr_pages* c) { return c->cfg; }
int kvr::pages_device(const kvr_pages* c) { return c->device; }
int kvr::pages_rows(const kvr_pages* c) { return c->rows; }

extern "C" {

size_t kvr_pages_pool_bytes(const kvr_pages_config* c) {
  if (!valid(c)) return 0;
  return (size_t)c->n_layers * c->n_pages * c->n_kv_heads * page_chunk_bytes(c->head_dim);
}

size_t kvr_pages_work_bytes(const kvr_pages_config* c) { return valid(c) ? layout(c).total : 0; }

int kvr_pages_create(const kvr_pages_config* cfg, void* pool, size_t pool_bytes, void* work, size_t work_bytes,
                     kvr_pages** out) {
  if (!out) return KVR_ERR_ARG;
  *out = nullptr;
  if (!valid(cfg) || !pool || !work || ((uintptr_t)pool & 255) || ((uintptr_t)work & 255)) return KVR_ERR_ARG;
  const Layout L = layout(cfg);
  if (pool_bytes < kvr_pages_pool_bytes(cfg) || work_bytes < L.total) return KVR_ERR_CAPACITY;
  kvr_pages* c = new (std::nothrow) kvr_pages();   // (no exception leaves a C entry)
  if (!c) return KVR_ERR_CAPACITY;
  c->cfg = *cfg;
  uint8_t* w = static_cast<uint8_t*>(work);
  PagesDev& d = c->dev;
  memset(&d, 0, sizeof d);
  d.pool = static_cast<uint8_t*>(pool);
  d.table = reinterpret_cast<int32_t*>(w + L.table);
  d.lens = reinterpret_cast<int32_t*>(w + L.lens);
  d.free_list = reinterpret_cast<int32_t*>(w + L.free_list);
  d.count = reinterpret_cast<int32_t*>(w + L.count);
  d.cu = reinterpret_cast<int32_t*>(w + L.cu);
  d.row_seq = reinterpret_cast<int32_t*>(w + L.row_seq);
  d.row_pos = reinterpret_cast<int32_t*>(w + L.row_pos);
  d.row_slot = reinterpret_cast<int32_t*>(w + L.row_slot);
  d.info = reinterpret_cast<int32_t*>(w + L.info);
  d.rope = reinterpret_cast<const float2*>(w + L.rope);
  d.rope_rest = reinterpret_cast<const __half2*>(w + L.rope_rest);
  d.status = reinterpret_cast<int*>(w + L.status);
  d.refused = d.status + 1;
  d.n_pages = cfg->n_pages;
  d.width = L.width;
  d.max_len = cfg->max_len;
  d.max_rows = cfg->max_rows;
  d.Hq = cfg->n_q_heads;
  d.Hkv = cfg->n_kv_heads;
  d.G = d.Hq / d.Hkv;
  d.d = cfg->head_dim;
  d.max_seqs = cfg->max_seqs;
  auto mul = [](int x) { return x == 1 ? 0u : (uint32_t)(((1ull << 32) + x - 1) / x); };
  d.mul_hkv = mul(d.Hkv);
  d.mul_g = mul(d.G);
  d.f16 = cfg->act == KVR_ACT_F16;
  c->layer_bytes = (size_t)cfg->n_pages * cfg->n_kv_heads * page_chunk_bytes(cfg->head_dim);
  memset(&c->attend, 0, sizeof c->attend);
  c->attend.part = reinterpret_cast<float*>(w + L.part);
  c->attend.ml = reinterpret_cast<float2*>(w + L.ml);
  c->attend.counters = reinterpret_cast<int*>(w + L.counters);
  memset(&c->attend_tc, 0, sizeof c->attend_tc);
  c->attend_tc.part = reinterpret_cast<float*>(w + L.part_tc);
  c->attend_tc.ml = reinterpret_cast<float2*>(w + L.ml_tc);
  c->attend_tc.shared = reinterpret_cast<PageShared*>(w + L.shared);
  int sms = 0;
  cudaError_t e = cudaGetDevice(&c->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, c->device);
  c->ctas = std::min(sms, kPageAttnMaxCtas);
  if (e == cudaSuccess) e = page_plan_setup();
  if (e == cudaSuccess) e = page_attn_setup();
  if (e == cudaSuccess) e = page_attn_tc_setup();
  if (e == cudaSuccess) e = cudaMemset(w + L.status, 0, L.count - L.status);
  if (e == cudaSuccess) e = cudaMemset(w + L.table, 0xff, (size_t)cfg->max_seqs * L.width * 4);
  if (e == cudaSuccess) e = cudaMemset(w + L.row_seq, 0xff, L.table - L.row_seq);
  if (e == cudaSuccess) e = launch_page_init(d, nullptr);
  if (e == cudaSuccess)
    e = launch_page_rope(rope_freq(cfg->rope_theta, cfg->head_dim), cfg->max_len, cfg->head_dim,
                         reinterpret_cast<float2*>(w + L.rope), reinterpret_cast<__half2*>(w + L.rope_rest), nullptr);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    delete c;
    return KVR_ERR_CUDA;
  }
  *out = c;
  return KVR_OK;
}

int kvr_pages_destroy(kvr_pages* c) {
  if (!c) return KVR_ERR_ARG;
  delete c;
  return KVR_OK;
}

int kvr_pages_tables(const kvr_pages* c, kvr_page_tables* out) {
  if (!c || !out) return KVR_ERR_ARG;
  const PagesDev& d = c->dev;
  *out = {d.table, d.lens, d.free_list, d.count, d.cu, d.row_seq, d.row_pos, d.row_slot, d.width};
  return KVR_OK;
}

int kvr_page_plan(kvr_pages* c, int n_seq, const int32_t* keep, const int32_t* add, int rows, int max_add,
                  void* stream) {
  if (!c) return KVR_ERR_ARG;
  if (n_seq < 1 || n_seq > c->cfg.max_seqs)
    return fail(c, KVR_ERR_ARG, "%d sequences outside [1, %d]", n_seq, c->cfg.max_seqs);
  if (!keep || !add || ((uintptr_t)keep & 3) || ((uintptr_t)add & 3))
    return fail(c, KVR_ERR_ARG, "keep and add must be device int32 arrays");
  if (rows < 0 || rows > c->cfg.max_rows)
    return fail(c, KVR_ERR_CAPACITY, "%d rows outside [0, %d]", rows, c->cfg.max_rows);
  if (max_add <= 0 || max_add > rows) max_add = rows;
  OnDevice on(c->device);
  const cudaError_t e =
      launch_page_plan(c->dev, n_seq, keep, add, rows, max_add, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(c, e, "page plan launch");
  c->rows = rows;
  c->max_add = max_add;
  c->n_seq = n_seq;
  return KVR_OK;
}

int kvr_page_append(kvr_pages* c, int layer, const void* q, long long q_stride, const void* k, long long k_stride,
                    const void* v, long long v_stride, const void* norm_q, const void* norm_k, int rotate,
                    void* q_out, int rows, void* stream) {
  if (!c) return KVR_ERR_ARG;
  PagesDev d;
  if (int rc = layer_call(c, layer, rows, &d)) return rc;
  if (rows == 0) return KVR_OK;
  if (!k || !v || (q == nullptr) != (q_out == nullptr)) return fail(c, KVR_ERR_ARG, "null q, k or v pointer");
  for (const void* p : {q, k, v, norm_q, norm_k, static_cast<const void*>(q_out)})
    if (!aligned(p)) return fail(c, KVR_ERR_ARG, "pointers must be 16-byte aligned");
  const long long qr = (long long)d.Hq * d.d, kr = (long long)d.Hkv * d.d;
  if ((q && !stride_ok(q_stride, qr)) || !stride_ok(k_stride, kr) || !stride_ok(v_stride, kr))
    return fail(c, KVR_ERR_ARG, "row strides must cover a row and be multiples of 8");
  if (q && q == q_out && q_stride != qr) return fail(c, KVR_ERR_ARG, "q_out may be q only if q's rows are contiguous");
  const long long q_bytes = 2 * qr * rows;
  if (q && ((q != q_out && overlap(q, 2 * q_stride, rows, 2 * qr, q_out, q_bytes)) ||
            overlap(k, 2 * k_stride, rows, 2 * kr, q_out, q_bytes) ||
            overlap(v, 2 * v_stride, rows, 2 * kr, q_out, q_bytes)))
    return fail(c, KVR_ERR_ARG, "q_out shares memory with k, v or other rows of q");
  const PageAppend a = {q,      k,     v,      q_stride,   k_stride, v_stride, norm_q,
                        norm_k, q_out, rotate, rows, c->cfg.norm_eps};
  OnDevice on(c->device);
  const cudaError_t e = launch_page_append(d, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVR_OK : cuda_fail(c, e, "page append launch");
}

int kvr_page_read(kvr_pages* c, int layer, void* k_out, void* v_out, int rows, void* stream) {
  if (!c) return KVR_ERR_ARG;
  PagesDev d;
  if (int rc = layer_call(c, layer, rows, &d)) return rc;
  if (rows == 0) return KVR_OK;
  if (!k_out || !v_out || !aligned(k_out) || !aligned(v_out))
    return fail(c, KVR_ERR_ARG, "missing or misaligned output pointer");
  const long long kr = 2ll * d.Hkv * d.d;
  if (overlap(k_out, kr, rows, kr, v_out, kr * rows)) return fail(c, KVR_ERR_ARG, "k_out and v_out share memory");
  OnDevice on(c->device);
  const cudaError_t e = launch_page_read(d, k_out, v_out, rows, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVR_OK : cuda_fail(c, e, "page read launch");
}

int kvr_page_attend(kvr_pages* c, int layer, const void* q, long long q_stride, void* out, int out_f16, float scale,
                    int rows, void* stream) {
  if (!c) return KVR_ERR_ARG;
  PagesDev d;
  if (int rc = layer_call(c, layer, rows, &d)) return rc;
  if (rows == 0) return KVR_OK;
  if (!q || !out || !aligned(q) || !aligned(out))
    return fail(c, KVR_ERR_ARG, "missing or misaligned q or out pointer");
  const long long qr = (long long)d.Hq * d.d;
  if (!stride_ok(q_stride, qr))
    return fail(c, KVR_ERR_ARG, "the row stride must cover a row and be a multiple of 8");
  if (overlap(q, 2 * q_stride, rows, 2 * qr, out, 2 * qr * rows)) return fail(c, KVR_ERR_ARG, "out shares memory with q");
  const float scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!(scale > 0.f) || !std::isfinite(scale_log2))
    return fail(c, KVR_ERR_ARG, "scale must be a positive number of at most 2.3e38");
  PageAttend a = c->attend;
  a.q = q;
  a.qs = q_stride;
  a.out = out;
  a.out_f16 = out_f16 || d.f16;
  a.rows = rows;
  a.scale_log2 = scale_log2;
  const long long most = (long long)d.G * c->max_add;   // rows of a sequence and KV head, at most
  const long long tiles = ((long long)d.G * rows + 7) / 8 + c->n_seq;   // of 8 rows, at most
  const bool few = tiles * d.width * d.Hkv <= (long long)kPageFew * c->ctas;
  const bool split_only = few || most <= kPageMany;
  a.many = !split_only ? kPageManyBeside : (int)std::max<long long>(most, kPageMany);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  OnDevice on(c->device);
  cudaError_t e = cudaSuccess;
  if (!split_only) {
    PageAttendTc b = c->attend_tc;
    b.q = q;
    b.qs = q_stride;
    b.out = out;
    b.out_f16 = a.out_f16;
    b.rows = rows;
    b.many = a.many;
    b.min_units = kPageMinUnits;
    b.scale_log2 = a.scale_log2;
    e = launch_page_attn_tc(d, b, c->ctas, st);
    if (e != cudaSuccess) return cuda_fail(c, e, "page attention launch");
    a.shared = b.shared;
    a.tc_part = b.part;
    a.tc_ml = b.ml;
  }
  e = launch_page_attn(d, a, c->ctas, st);
  return e == cudaSuccess ? KVR_OK : cuda_fail(c, e, "page attention launch");
}

int kvr_pages_sync(kvr_pages* c, void* stream) {
  if (!c) return KVR_ERR_ARG;
  OnDevice on(c->device);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int word[2] = {0, 0};
  cudaError_t e = cudaMemcpyAsync(word, c->dev.status, 8, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && (word[0] || word[1])) {
    e = cudaMemsetAsync(c->dev.status, 0, 8, st);
    // a launch that gave up may have left arrivals behind
    if (e == cudaSuccess && word[0]) e = cudaMemsetAsync(c->attend.counters, 0, kPageAttnMaxCtas * 4, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  if (e != cudaSuccess) return cuda_fail(c, e, "page status readback");
  if (word[0]) return fail(c, KVR_ERR_TIMEOUT, "a device-side wait gave up (status %d)", word[0]);
  if (word[1] == KVR_ERR_CAPACITY) return fail(c, KVR_ERR_CAPACITY, "a plan lacked free pages and was not carried out");
  if (word[1] == KVR_ERR_UNSUPPORTED)
    return fail(c, KVR_ERR_ARG, "an attend was captured under a smaller max_add than its step's; rows were left out");
  if (word[1]) return fail(c, KVR_ERR_ARG, "a plan's keep or add were out of range; it was not carried out");
  return KVR_OK;
}

const char* kvr_pages_error(const kvr_pages* c) { return c ? c->err : "null handle"; }

}  // extern "C"
