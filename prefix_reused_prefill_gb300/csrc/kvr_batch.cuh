// Internal declarations of what the requests of one batch differ by: sampling
// and low-rank adapters (include/kvr.h).
#pragma once

#include "kvr_internal.cuh"

namespace kvr {

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

cudaError_t launch_sample(const SampleParams& p, int sms, cudaStream_t st);

}  // namespace kvr
