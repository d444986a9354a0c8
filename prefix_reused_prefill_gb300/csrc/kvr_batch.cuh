// Internal declarations of what the requests of one batch differ by: sampling
// and low-rank adapters (include/kvr.h).
#pragma once

#include "kvr_internal.cuh"

namespace kvr {

// Rows of memory: n of `width` bytes, `stride` bytes apart (one row: any).
struct Span {
  const void* p;
  long long n, stride, width;
  Span(const void* p_, long long width_) : p(p_), n(1), stride(width_), width(width_) {}
  Span(const void* p_, long long n_, long long stride_, long long width_) : p(p_), n(n_), stride(stride_), width(width_) {}
  long long bytes() const { return (n - 1) * stride + width; }
};
// Whether two of them share a byte.  (Rows that stand among one another at different strides count as
// sharing.)
bool shared(const Span& a, const Span& b);

constexpr int kSampleIndexBits = 18;   // KVR_MAX_VOCAB = 2^18
static_assert(KVR_MAX_VOCAB <= 1 << kSampleIndexBits, "a token's index has to fit beside its logit");

struct SampleParams {
  const void* logits;       // [rows], stride elements apart
  long long stride;
  int rows, vocab, type;    // KVR_ACT_*
  kvr_sampling s;           // per row, or per sequence where cu is given
  const float* u;           // [rows]
  // kvr_sample
  int32_t* token;           // [rows]
  float* prob;              // [rows] or null
  float* dist;              // [rows] dist_stride apart, or null
  long long dist_stride;
  // kvr_accept (cu not null)
  const int32_t* cu;        // [n_seq + 1]
  int n_seq;
  const int32_t* tokens;    // [rows]
  const float* q;           // [rows] q_stride apart, or null
  long long q_stride;
  const float* u_next;      // [n_seq]
  int32_t* outcome;         // [rows] kStays, or the token that follows
  int32_t *accepted, *next; // [n_seq]
};
constexpr int kStays = -2;

cudaError_t sample_setup();   // of the current device, before its first launch
cudaError_t launch_sample(const SampleParams& p, int sms, cudaStream_t st);

constexpr int kAdaptMaxSeqs = 2048;
constexpr int kAdaptMaxSplit = 48;
constexpr int kAdaptRows = 8;        // rows of a tile
struct AdaptParams {
  kvr_adapter_site site;
  const void* x;
  long long x_stride;
  int x16;                 // x is fp16 that holds the site's bf16 values
  const int32_t *cu, *which;
  int n_seq, rows;
  const void* base;        // or null
  long long base_stride;
  void* out;
  long long out_stride;
  int out_type;
  float* part;             // [ksplit][rows][n_parts * max_rank] parts of the low-rank products
  int ksplit;
  int* status;             // of a context, or the device's (adapt_status): a wait that gave up
};
cudaError_t adapt_setup();    // of the current device, before its first launch
cudaError_t adapt_status(int** word);   // where the current device's word is
bool adapter_site_ok(const kvr_adapter_site* s);
size_t adapt_work_bytes(const kvr_adapter_site& s, int rows);
cudaError_t launch_adapt(AdaptParams p, int sms, cudaStream_t st);

}  // namespace kvr
