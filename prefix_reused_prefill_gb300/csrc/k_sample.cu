// Sampling from given random numbers, and speculative sampling (include/kvr.h).
//
// A row's tokens are never sorted.  Everything asked of their order is of one kind:
// the shortest run from the largest logit that holds a count (top_k) or a weight
// (top_p; the drawn token ends the run that holds more than u of the weight).  So
// one pass files the tokens under their logit's distance from the maximum, in bins
// of 1/32 of a binary order that hold the count and the weight; running sums over
// the bins name the bin in which a run ends, and only the tokens up to it, where
// they are few, or that bin's are put in order.
//
// The bins hold 32 binary orders at a time: what is further from the maximum is summed
// in registers, and filed in a later pass only if a run ends there.  Where top_k
// bounds the kept tokens the first pass only counts.
//
// A token's place is one 50-bit number, its logit's bits above its inverted
// index, so equal logits need no care.  Weights are formed to 2^-46 in pairs
// of floats and summed as whole numbers of 2^-44 of the largest: whole numbers have
// one sum in any order, so shared-memory atomics serve and every pass, CTA and
// launch agrees on where a run ends.
//
// A row is a cluster's, of up to eight CTAs; each files its share of the tokens in
// shared memory, the first one adds the bins up through distributed shared memory and
// searches.  What bounds it is not the logits' way from memory (a pass over 33 MB of
// them takes 5 us) but arithmetic: about a hundred instructions a token, most of them for
// the weight.  One CTA files 32768 tokens in 12 us, two on an SM in 24.  The passes of
// a row of 262144 tokens: maximum 4 us, bins 12, their sums and the search 4, and for
// each end of a run that more than 2048 tokens stand before, 2 to 7 us of a pass that
// looks up one bin's tokens and 3 that orders them.
// Per call in a graph: one row of 32000 10.5 us, 64 rows of 131072 with different
// settings 57, 16 rows of 262144 without any bound 55 (15 clusters of eight fit alone; where two share their SMs
// the passes take twice as long).
#include <cooperative_groups.h>

#include <type_traits>
#include <utility>

#include "kvr_batch.cuh"

namespace cg = cooperative_groups;

namespace kvr {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512;        // (with 1024 a row's CTAs do not all run at once, and it took longer)
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;          // held at a time, two a thread
constexpr int kFix = 44;
constexpr float kNothing = 46.f;     // binary orders from the maximum on which a token weighs nothing
// Steps (1/1024 of a binary order) of a bin, by their logarithm: where weights are filed 32, so that
// 32 orders are held at a time and a bin of the bulk of 262144 tokens is about as many as can be put
// in order; where tokens are only counted 64, so that one pass holds all.
constexpr int kFine = 5, kCoarse = 6;
constexpr int kCap = 2048;           // tokens that one CTA puts in order
constexpr int kCount = 128;          // as many by counting the larger ones
constexpr int kPart = 64;            // tokens of one part of a list from which on the list is sorted instead
constexpr int kDigit = 10;           // bits of a place taken at a time where a bin holds more
static_assert(kBins == 2 * kThreads && kBins == 1 << kDigit && kCount <= kThreads && (kCap & (kCap - 1)) == 0, "bins and digits two a thread");
constexpr int kPlaceBits = 32 + kSampleIndexBits;
constexpr uint32_t kIndexMask = (1u << kSampleIndexBits) - 1;

// 2^(-i/1024) as a pair of floats, from the exponential series.
struct Pow2Table {
  float hi[1024], lo[1024];
};
constexpr Pow2Table pow2_table() {
  Pow2Table t{};
  for (int i = 0; i < 1024; ++i) {
    const double z = -0.69314718055994530942 * i / 1024;
    double term = 1, sum = 0;
    for (int k = 1; k < 24; ++k) {
      sum += term;
      term *= z / k;
    }
    t.hi[i] = (float)sum;
    t.lo[i] = (float)(sum - (double)t.hi[i]);
  }
  return t;
}
__device__ const Pow2Table kPow2 = pow2_table();

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

struct Bins {
  uint32_t cnt[kBins + 32], lo[kBins + 32], hi[kBins + 32];   // (Sampler::add; two of each, by lane, were slower)
};
struct Smem {
  float2 pow2[1024];
  Bins bins;
  u64 mine[kCap];           // this CTA's tokens of a bin
  int filled;               // how many
  u64 front_w, rest_w;      // this CTA's tokens in front of the bins and behind them
  uint32_t front_c, rest_c;
  double min_orders;        // temperature * ln(min_p)
  // what the cluster's CTAs tell one another
  uint32_t best_key[kMaxCluster], best_i[kMaxCluster];
  u64 warp_w[kWarps];
  uint32_t warp_c[kWarps], warp_i[kWarps];
  // of the cluster's first CTA: running weights and counts over the bins and over the parts of one bin,
  // those of the row, and the tokens to be put in order
  u64 sum_w[kBins], part_w[kBins];
  uint32_t sum_c[kBins], part_c[kBins];
  u64 before_w, total_w;
  uint32_t before_c, total_c;
  u64 place[kCap], weight[kCap];
  int bin, n;               // the bin in which a run ends and its tokens; kLower, kHigher: not in these
  u64 base_w;               // weight and count in front of it
  uint32_t base_c;
  u64 from;                 // first place of a part of it
  u64 run_place, run_w;     // the end of a run, its weight
  u64 kept, kept_w;         // the row's distribution
  int found, stays;
};
constexpr int kLower = -1, kHigher = -2;

// Two floats in one register pair, and the instructions that take them (each rounded as alone).
__device__ __forceinline__ u64 two(float lo, float hi) {
  u64 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ u64 two(float x) { return two(x, x); }
__device__ __forceinline__ void split(u64 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ u64 sub2(u64 a, u64 b) { return fma2(b, two(-1.f), a); }

// What a row's tokens weigh.
constexpr float kFinite = 3.4028234663852886e38f;
struct Row {
  float max;            // (where it is infinite, the largest number: `floor` then leaves the infinite ones)
  float ch, cl;         // log2(e) / temperature
  float floor;          // logits below weigh less than min_p
  // of a rejected draft's row: weight beyond the drafter's
  const float* q;       // null: all weight of `draft` goes
  u64 total;            // of p, its first bit the highest; (zeros in front) + 126
  int total_low;
  int draft;
  bool draft_in;        // within the vocabulary; its logit
  float draft_x;
  u64 kept;             // places from here on
  bool rest;

  __device__ __forceinline__ void set_total(u64 t) {
    const int zeros = __clzll((long long)t);
    total = t << zeros;
    total_low = zeros + 126;
  }
  // q total, to the next whole number (nothing for what is not a probability; in whole numbers, as 64-bit floats
  // run at a thirtieth of their rate here: 40 us for a row's 32768 tokens)
  __device__ __forceinline__ u64 taken(float q) const {
    if (!(q >= 0x1p-126f)) return 0;
    const uint32_t b = __float_as_uint(q), m = (b << 8) | 0x80000000u;
    const u64 prod = (u64)(uint32_t)(total >> 32) * m + __umulhi((uint32_t)total, m);
    const int s = total_low - (int)(b >> 23);
    if (s <= 0) return s < 0 ? ~0ull : prod;   // (below: q above 1)
    if (s > 64) return 0;
    return (s < 64 ? prod >> s : 0) + ((prod >> (s - 1)) & 1);
  }

  // binary orders below the maximum, as a pair (of what is at infinity only the
  // first number counts)
  __device__ __forceinline__ void orders(float x, float& yh, float& yl) const {
    x = fminf(x, kFinite);
    const float d = max - x;
    const float b = d - max;
    const float dl = (max - (d - b)) - (x + b);
    yh = d * ch;
    yl = fmaf(d, ch, -yh) + fmaf(d, cl, dl * ch);
  }
  // two at once
  __device__ __forceinline__ void orders(u64 x, u64& yh, u64& yl) const {
    const u64 m = two(max);
    const u64 d = sub2(m, x);
    const u64 b = sub2(d, m);
    const u64 dl = sub2(sub2(m, sub2(d, b)), add2(x, b));
    yh = mul2(d, two(ch));
    yl = add2(fma2(d, two(ch), mul2(d, two(-ch))), fma2(d, two(cl), mul2(dl, two(ch))));
  }
};

__device__ __forceinline__ u64 place_of(float x, int i) {
  const uint32_t b = __float_as_uint(x + 0.f);   // (-0 is 0)
  const uint32_t k = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  return ((u64)k << kSampleIndexBits) | (kIndexMask - (uint32_t)i);
}

__device__ __forceinline__ float logit_of(u64 place) {
  const uint32_t k = (uint32_t)(place >> kSampleIndexBits);
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ int token_of(u64 place) { return (int)(kIndexMask - (uint32_t)(place & kIndexMask)); }

// 2^-(yh + yl) = (s + r) 2^-n for distances of any size, as below.
__device__ __forceinline__ void pow2_neg(const float2* tab, float yh, float yl, float& s, float& r, int& n) {
  constexpr float kLn2h = 0.693147182464599609375f;
  constexpr float kLn2l = -1.904654323148236e-09f;
  const int j = __float2int_rd(yh * 1024.f);
  const float f = fmaf((float)j, -1.f / 1024.f, yh);
  const float zh = -f * kLn2h;
  const float zl = fmaf(-f, kLn2h, -zh) - fmaf(f, kLn2l, yl * kLn2h);
  const float e = fmaf(zh * zh, fmaf(zh, fmaf(zh, 1.f / 24.f, 1.f / 6.f), 0.5f), zl);
  const float2 t = tab[j & 1023];
  n = j >> 10;
  const float a = t.x * zh;
  float al = fmaf(t.x, zh, -a);
  al = fmaf(t.y, zh, al) + fmaf(t.x, e, t.y);
  s = t.x + a;
  r = (a - (s - t.x)) + al;
}

// the larger of two, NaN if one is
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// Distances in steps of 1/1024 of an order: the low bits of the float that has a
// step as its unit.  Distances of 64 orders and more count as the last bin's.
constexpr float kStepOne = 12582912.f;   // 1.5 * 2^23
constexpr uint32_t kStepBin = 0x4b400000u >> kFine;   // (its bits: the steps are added to them)
__device__ __forceinline__ uint32_t steps_of(float yh) {
  return __float_as_uint(fmaf(fminf(yh, 63.96875f), 1024.f, kStepOne)) - __float_as_uint(kStepOne);
}

// Two weights in units of 2^-44, as 2^-(yh + yl) = (s + r) 2^-n with the nearest
// step from the table and the rest by its series, whose first term is a pair of
// floats; yh in [0, 63.96875] (`steps`: those of yh, as above, with the float's own bits).
__device__ __forceinline__ void weights_of_two(const float2* tab, u64 yh, u64 yl, u64 steps, u64& v0, u64& v1) {
  constexpr float kLn2h = 0.693147182464599609375f;
  constexpr float kLn2l = -1.904654323148236e-09f;
  const u64 f = fma2(add2(steps, two(-kStepOne)), two(-1.f / 1024.f), yh);
  const u64 zh = mul2(f, two(-kLn2h)), zn = mul2(f, two(kLn2h));
  const u64 zl = sub2(fma2(f, two(-kLn2h), zn), fma2(f, two(kLn2l), mul2(yl, two(kLn2h))));
  const u64 e = fma2(mul2(zh, zh), fma2(zh, two(1.f / 6.f), two(0.5f)), zl);   // (z^4 / 24 is below 2^-50)
  const uint32_t j0 = (uint32_t)steps, j1 = (uint32_t)(steps >> 32);
  const float2 t0 = tab[j0 & 1023], t1 = tab[j1 & 1023];
  const u64 px = two(t0.x, t1.x), py = two(t0.y, t1.y);
  const u64 a = mul2(px, zh);
  const u64 s = add2(px, a);
  const u64 rest = add2(fma2(py, zh, fma2(px, zh, mul2(px, zn))), fma2(px, e, py));
  const u64 r = add2(sub2(a, sub2(s, px)), rest);
  float s0, s1, r0, r1;
  split(mul2(s, two(0x1p30f)), s0, s1);
  split(mul2(r, two(0x1p45f)), r0, r1);
  const auto whole = [](float s, float r, uint32_t j) {
    // (in half units, and to the nearest unit: weights of a few units may be all that a rejected draft leaves)
    const long long v = (long long)__float2int_rn(s) * (1ll << (kFix - 29)) + __float2int_rn(r);
    return (((u64)v >> ((j >> 10) & 63)) + 1) >> 1;
  };
  v0 = whole(s0, r0, j0);
  v1 = whole(s1, r1, j1);
}

// One of them.  (One arithmetic: wherever a token is weighed it weighs the same.)
__device__ __forceinline__ u64 weight_fixed(const float2* tab, float yh, float yl) {
  yh = fminf(yh, 63.96875f);
  u64 v0, v1;
  weights_of_two(tab, two(yh), two(yl), two(fmaf(yh, 1024.f, kStepOne)), v0, v1);
  return v0;
}

// total as a pair of floats
__device__ __forceinline__ float2 pair_of(u64 total) {
  const float h = __ull2float_rn(total);
  return make_float2(h * 0x1p-44f, __ll2float_rn((long long)(total - __float2ull_rn(h))) * 0x1p-44f);
}
// (s + r) 2^-n / total, rounded to a float but for 2^-46 of it
__device__ __forceinline__ float share_of(float s, float r, int n, float2 total) {
  const float q = s / total.x;
  const float v = q + (fmaf(-q, total.x, s) + fmaf(-q, total.y, r)) / total.x;
  // (in two steps, of which only the second may leave the normal numbers)
  const int m = min(n, 100);
  return v * __int_as_float((127 - m) << 23) * __int_as_float((127 - (n - m)) << 23);
}

// A CTA's tokens [lo, hi) of a row, four at a time where they are aligned to it.
template <class T>
struct Tokens {
  const T* row;
  int lo, hi, a, fours, items;
  __device__ __forceinline__ Tokens(const T* row_, int lo_, int hi_) : row(row_), lo(lo_), hi(hi_) {
    constexpr int kBytes = 4 * sizeof(T);
    const int skip = (int)((kBytes - ((uintptr_t)(row + lo) & (kBytes - 1))) & (kBytes - 1)) / (int)sizeof(T);
    a = min(lo + skip, hi);
    fours = (hi - a) / 4;
    items = fours + (hi - lo - 4 * fours);
  }
  // item t: its tokens from i on, n of them (4, or 1)
  __device__ __forceinline__ void load(int t, float (&x)[4], int& i, int& n) const {
    if (t < fours) {
      i = a + 4 * t;
      n = 4;
      typename std::conditional<sizeof(T) == 4, uint4, uint2>::type v;
      v = *reinterpret_cast<const decltype(v)*>(row + i);
      const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = to_float(e[k]);
    } else {
      const int left = t - fours;
      i = left < a - lo ? lo + left : a + 4 * fours + left - (a - lo);
      n = 1;
      x[0] = to_float(row[i]);
      x[1] = x[2] = x[3] = __int_as_float(0x7fffffff);   // (NaN: never one of a row's)
    }
  }
};

// f(logits, token of the first, how many) over the CTA's tokens, U times four in flight.
template <int U, class T, class F>
__device__ __forceinline__ void for_tokens(const T* row, int lo, int hi, F f) {
  const Tokens<T> tk(row, lo, hi);
  int t = threadIdx.x;
  float x[U][4];
  int i[U], n[U];
  if constexpr (U == 1) {
    // (much to do for each: one copy of it, the next four on their way)
    if (t < tk.items) tk.load(t, x[0], i[0], n[0]);
    while (t < tk.items) {
      float y[4];
      int j = 0, m = 0;
      if (t + kThreads < tk.items) tk.load(t + kThreads, y, j, m);
      f(x[0], i[0], n[0]);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[0][k] = y[k];
      i[0] = j;
      n[0] = m;
      t += kThreads;
    }
  } else {
    for (; t < tk.items; t += U * kThreads) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        n[k] = 0;
        if (t + k * kThreads < tk.items) tk.load(t + k * kThreads, x[k], i[k], n[k]);
      }
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (n[k]) f(x[k], i[k], n[k]);
    }
  }
}

// ceil(total * p) and floor(total * u) + 1 for p, u in [0, 1), exactly
__device__ __forceinline__ u64 share(u64 total, float p, bool up) {
  const int e = ilogbf(p) - 23;                             // p = m 2^e
  const u64 m = (u64)__float2ull_rn(scalbnf(p, -e));        // (24 bits)
  if (p == 0.f || e < -120) return up ? (p == 0.f ? 0 : 1) : 1;
  const u64 hi = __umul64hi(total, m), lo = total * m;
  const int s = -e;                                         // 24 .. 120
  u64 whole, left;
  if (s < 64) {
    whole = (hi << (64 - s)) | (lo >> s);
    left = lo << (64 - s);
  } else {
    whole = s == 64 ? hi : hi >> (s - 64);
    left = (s == 64 ? 0 : hi << (128 - s)) | lo;
  }
  return whole + (up ? left != 0 : 1);
}

// Sums and searches over n ordered weights, four a thread: by one warp, or by the CTA.
constexpr int kPer = kCap / kThreads;
template <int THREADS>
struct Scan {
  Smem& sm;
  int at, n;
  u64 v[kPer], before;
  __device__ __forceinline__ int entry(int k) const { return (threadIdx.x % THREADS) * kPer + k; }
  __device__ __forceinline__ static void sync() {
    if (THREADS == 32) __syncwarp();
    else __syncthreads();
  }
  __device__ __forceinline__ void sum() {
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[k] = (entry(k) < n ? sm.weight[at + entry(k)] : 0) + (k ? v[k - 1] : 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 r = v[kPer - 1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 a = __shfl_up_sync(0xffffffffu, r, o);
      if (lane >= o) r += a;
    }
    before = r - v[kPer - 1];
    if (THREADS == 32) return;
    __syncthreads();
    if (lane == 31) sm.warp_w[warp] = r;
    __syncthreads();
    for (int k = 0; k < warp; ++k) before += sm.warp_w[k];
  }
  __device__ __forceinline__ u64 total() {
    if (THREADS == 32) return __shfl_sync(0xffffffffu, before + v[kPer - 1], 31);
    if (threadIdx.x == kThreads - 1) sm.run_w = before + v[kPer - 1];
    __syncthreads();
    const u64 t = sm.run_w;
    __syncthreads();
    return t;
  }
  // the entry at which the weight reaches `mass`, and the weight there
  __device__ __forceinline__ int reach(u64 mass, u64& weight) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const u64 iw = before + v[k], pw = before + (k ? v[k - 1] : 0);
      if (entry(k) < n && iw >= mass && pw < mass) {
        sm.found = entry(k);
        sm.run_w = iw;
      }
    }
    sync();
    const int i = min(max(sm.found, 0), max(n - 1, 0));   // (an entry, whatever the weights were)
    weight = sm.run_w;
    sync();
    return i;
  }
};

// n numbers (a power of two of them) into descending order, by compare and exchange (2048: in 66 steps).
__device__ __forceinline__ void sort_list(u64* list, int n) {
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int t = threadIdx.x; t < n / 2; t += kThreads) {
        const int i = 2 * t - (t & (j - 1));
        const u64 a = list[i], b = list[i + j];
        if ((a < b) == ((i & k) == 0)) {
          list[i] = b;
          list[i + j] = a;
        }
      }
      __syncthreads();
    }
}

template <class T>
struct Sampler {
  Smem& sm;
  Smem& first;          // the cluster's first CTA's
  const cg::cluster_group& cluster;
  const T* row;
  int lo, hi;           // this CTA's tokens
  int rank, ctas;
  Row w;
  int shift;            // log2 of the steps of a bin
  int bin0;             // the first one held

  // (bins are told apart by the logit's distance alone, so equal logits share one)
  __device__ __forceinline__ int bin_of(float yh) const { return (int)(steps_of(yh) >> shift); }

  // A token's weight: what a draft left of it, where the row is such a one.
  __device__ __forceinline__ u64 weigh(int i, float yh, float yl) const {
    return yh < kNothing ? left(weight_fixed(sm.pow2, yh, yl), i) : 0;
  }
  __device__ __forceinline__ u64 left(u64 v, int i) const {
    if (!w.rest) return v;
    if (!w.q) return i == w.draft ? 0 : v;
    const u64 t = w.taken(w.q[i]);
    return v > t ? v - t : 0;
  }
  // whether a token is one of the row's
  __device__ __forceinline__ bool in_row(float x, int i) const {
    return x >= w.floor && (!w.rest || place_of(x, i) >= w.kept);
  }
  __device__ __forceinline__ void sync() {
    if (ctas > 1) cluster.sync();
    else __syncthreads();
  }

  __device__ __forceinline__ void clear_bins(bool mass) {
    uint4* b = reinterpret_cast<uint4*>(&sm.bins);
    const int n = (int)((mass ? sizeof(Bins) : sizeof(sm.bins.cnt)) / 16);
    for (int i = threadIdx.x; i < n; i += kThreads) b[i] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x == 0) {
      sm.front_w = sm.rest_w = 0;
      sm.front_c = sm.rest_c = 0;
    }
    __syncthreads();
  }
  // N tokens into their bins (< 0: none), without a branch and the atomics in flight
  // together: a lane has a bin of its own for what goes nowhere.
  template <int N>
  __device__ __forceinline__ void add(const int (&bin)[N], const u64 (&v)[N]) const {
    const int none = kBins + (threadIdx.x & 31);
    uint32_t old[N], at[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      at[k] = bin[k] >= 0 ? bin[k] : none;
      atomicAdd(&sm.bins.cnt[at[k]], 1u);
      old[k] = atomicAdd(&sm.bins.lo[at[k]], (uint32_t)v[k]);
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
      atomicAdd(&sm.bins.hi[at[k]], (uint32_t)(v[k] >> 32) + (old[k] + (uint32_t)v[k] < old[k] ? 1u : 0u));
  }

  // Running sums over the cluster's bins, after what is in front of them, to the
  // first CTA's sum_w and sum_c.  The others return once it may read theirs.
  template <bool MASS>
  __device__ __forceinline__ void sum_bins(u64* sum_w, uint32_t* sum_c, const u64* front_w, const uint32_t* front_c) {
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = 2 * threadIdx.x;
    u64 v[2] = {0, 0};
    uint32_t c[2] = {0, 0};
    {
      const uint2 n = *reinterpret_cast<const uint2*>(&sm.bins.cnt[b]);
      c[0] = n.x;
      c[1] = n.y;
      if (MASS) {
        const uint2 l = *reinterpret_cast<const uint2*>(&sm.bins.lo[b]);
        const uint2 h = *reinterpret_cast<const uint2*>(&sm.bins.hi[b]);
        v[0] = (u64)h.x << 32 | l.x;
        v[1] = (u64)h.y << 32 | l.y;
      }
    }
    if (ctas > 1) {
      cluster.sync();
      if (rank) return;
      // (all CTAs' on their way together; the first one stands in for those that there are not)
      uint2 n[kMaxCluster], l[kMaxCluster], h[kMaxCluster];
#pragma unroll
      for (int j = 1; j < kMaxCluster; ++j) {
        const Bins& o = cluster.map_shared_rank(&sm, j < ctas ? j : 0)->bins;
        n[j] = *reinterpret_cast<const uint2*>(&o.cnt[b]);
        if (MASS) {
          l[j] = *reinterpret_cast<const uint2*>(&o.lo[b]);
          h[j] = *reinterpret_cast<const uint2*>(&o.hi[b]);
        }
      }
#pragma unroll
      for (int j = 1; j < kMaxCluster; ++j)
        if (j < ctas) {
          c[0] += n[j].x;
          c[1] += n[j].y;
          if (MASS) {
            v[0] += (u64)h[j].x << 32 | l[j].x;
            v[1] += (u64)h[j].y << 32 | l[j].y;
          }
        }
    }
    if (front_w == &sm.before_w && warp == 0) {
      u64 fw = 0, rw = 0;
      uint32_t fc = 0, rc = 0;
      if (MASS && lane < ctas) {
        const Smem* o = cluster.map_shared_rank(&sm, lane);
        fw = o->front_w;
        rw = o->rest_w;
        fc = o->front_c;
        rc = o->rest_c;
      }
      if (MASS) {
        fc = __reduce_add_sync(0xffffffffu, fc);
        rc = __reduce_add_sync(0xffffffffu, rc);
#pragma unroll
        for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
          fw += __shfl_xor_sync(0xffffffffu, fw, o);
          rw += __shfl_xor_sync(0xffffffffu, rw, o);
        }
      }
      if (lane == 0) {
        sm.before_w = fw;
        sm.before_c = fc;
        sm.total_w = rw;
        sm.total_c = rc;
      }
    }
    v[1] += v[0];
    c[1] += c[0];
    u64 rv = v[1];
    uint32_t rc = c[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, rc, o);
      if (lane >= o) rc += y;
      if (MASS) {
        const u64 x = __shfl_up_sync(0xffffffffu, rv, o);
        if (lane >= o) rv += x;
      }
    }
    if (lane == 31) {
      sm.warp_c[warp] = rc;
      sm.warp_w[warp] = rv;
    }
    __syncthreads();
    u64 bv = *front_w + rv - v[1];
    uint32_t bc = *front_c + rc - c[1];
    for (int k = 0; k < warp; ++k) {
      bc += sm.warp_c[k];
      if (MASS) bv += sm.warp_w[k];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sum_w[b + k] = bv + v[k];
      sum_c[b + k] = bc + c[k];
    }
    if (front_w == &sm.before_w && threadIdx.x == kThreads - 1) {
      sm.total_w += bv + v[1];
      sm.total_c += bc + c[1];
    }
    __syncthreads();
  }

  // The row's tokens into the bins from `to` on, with their weights or only counted,
  // and the running sums (the first CTA's, until the next sync).
  template <bool MASS>
  __device__ __forceinline__ void file(int to) {
    bin0 = to;
    shift = MASS ? kFine : kCoarse;
    clear_bins(MASS);
    const Sampler c = *this;   // (in registers)
    u64 front_w = 0, rest_w = 0;
    uint32_t front_c = 0, rest_c = 0;
    for_tokens<1>(c.row, c.lo, c.hi, [&](const float (&x)[4], int i, int n) {
      constexpr int N = 4;
      if (!MASS) {
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (c.in_row(x[k], i + k))
            atomicAdd(&c.sm.bins.cnt[c.bin_of((c.w.max - fminf(x[k], kFinite)) * c.w.ch)], 1u);
        return;
      }
      u64 yh[N / 2], yl[N / 2], steps[N / 2];
      int b[N];
      float least = 64.f;
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        c.w.orders(two(fminf(x[k], kFinite), fminf(x[k + 1], kFinite)), yh[k / 2], yl[k / 2]);
        float y0, y1;
        split(yh[k / 2], y0, y1);
        y0 = fminf(y0, 63.96875f);
        y1 = fminf(y1, 63.96875f);
        least = fminf(least, fminf(y0, y1));
        yh[k / 2] = two(y0, y1);
        steps[k / 2] = fma2(yh[k / 2], two(1024.f), two(kStepOne));
        // (a token that is not the row's has bin -1; the others' are 0 and more)
        b[k] = x[k] >= c.w.floor ? (int)(((uint32_t)steps[k / 2] >> kFine) - kStepBin) : -1;
        b[k + 1] = x[k + 1] >= c.w.floor ? (int)(((uint32_t)(steps[k / 2] >> 32) >> kFine) - kStepBin) : -1;
      }
      u64 v[N] = {0, 0, 0, 0};
      if (least < kNothing) {
#pragma unroll
        for (int k = 0; k < N; k += 2)
          weights_of_two(c.sm.pow2, yh[k / 2], yl[k / 2], steps[k / 2], v[k], v[k + 1]);
      } else if (!c.bin0) {   // (far behind the first bins, and without weight)
#pragma unroll
        for (int k = 0; k < N; ++k) rest_c += b[k] >= 0 ? 1 : 0;
        return;
      }
      if (c.w.rest) {
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (b[k] >= 0) {
            if (place_of(x[k], i + k) < c.w.kept) b[k] = -1;
            else v[k] = c.left(v[k], i + k);
          }
      }
      if (c.bin0) {
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (b[k] >= 0) {
            b[k] -= c.bin0;
            if (b[k] < 0) {
              ++front_c;
              front_w += v[k];
            }
          }
      }
      if (max(max(b[0], b[1]), max(b[2], b[3])) >= kBins) {   // behind the bins
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (b[k] >= kBins) {
            b[k] = -1;
            ++rest_c;
            rest_w += v[k];
          }
      }
      c.add(b, v);
    });
    if (MASS) {
      front_c = __reduce_add_sync(0xffffffffu, front_c);
      rest_c = __reduce_add_sync(0xffffffffu, rest_c);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        if (bin0) front_w += __shfl_xor_sync(0xffffffffu, front_w, o);
        rest_w += __shfl_xor_sync(0xffffffffu, rest_w, o);
      }
      if ((threadIdx.x & 31) == 0) {
        if (front_c) atomicAdd(&sm.front_c, front_c);
        if (rest_c) atomicAdd(&sm.rest_c, rest_c);
        if (front_w) atomicAdd(&sm.front_w, front_w);
        if (rest_w) atomicAdd(&sm.rest_w, rest_w);
      }
    }
    sum_bins<MASS>(sm.sum_w, sm.sum_c, &sm.before_w, &sm.before_c);
  }

  // The bin (of those held, or of one bin's parts) in which the run that holds
  // `count` tokens or (count 0) `mass` ends.  First CTA only.
  __device__ __forceinline__ void find_bin(const u64* sum_w, const uint32_t* sum_c, u64 before_w, uint32_t before_c,
                                           uint32_t count, u64 mass, int offset) {
    if (threadIdx.x == 0) sm.bin = (count ? count <= before_c : mass <= before_w) ? kLower : kHigher;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int b = 2 * threadIdx.x + k;
      const u64 iw = sum_w[b], pw = b ? sum_w[b - 1] : before_w;
      const uint32_t ic = sum_c[b], pc = b ? sum_c[b - 1] : before_c;
      if (count ? ic >= count && pc < count : iw >= mass && pw < mass) {
        sm.bin = offset + b;
        sm.n = (int)(ic - pc);
        sm.base_w = pw;
        sm.base_c = pc;
      }
    }
    __syncthreads();
  }

  // Distances of bins b0 .. b1 (behind the last one nothing is): their bounds are floats.
  __device__ __forceinline__ float2 bounds(int b0, int b1) const {
    return make_float2(((float)(b0 << shift) - 0.5f) / 1024.f,
                       (b1 + 1) << shift < 65536 ? ((float)((b1 + 1) << shift) - 0.5f) / 1024.f
                                                 : __int_as_float(0x7fffffff));
  }
  // f(logit, token, place) for the CTA's tokens of bins b0 .. b1, in [from, from + 2^width) of their places
  template <class F>
  __device__ __forceinline__ void members(int b0, int b1, u64 from, int width, F f) const {
    const Sampler c = *this;   // (in registers)
    const float2 y = bounds(b0, b1);
    for_tokens<4>(c.row, c.lo, c.hi, [&](const float (&x)[4], int i, int m) {
      // (the nearest of the four first: most have nothing near enough)
      const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      if (!(top >= c.w.floor) || (c.w.max - fminf(top, kFinite)) * c.w.ch >= y.y) return;
      uint32_t hits = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float yh = (c.w.max - fminf(x[k], kFinite)) * c.w.ch;
        hits |= (!(yh < y.x) && !(yh >= y.y) && x[k] >= c.w.floor ? 1u : 0u) << k;
      }
      while (hits) {
        const int k = __ffs(hits) - 1;
        hits &= hits - 1;
        const float xk = k == 0 ? x[0] : k == 1 ? x[1] : k == 2 ? x[2] : x[3];
        const u64 p = place_of(xk, i + k);
        if (p >= from && !((p - from) >> width) && !(c.w.rest && p < c.w.kept)) f(xk, i + k, p);
      }
    });
  }
  // The tokens of bins b0 .. b1 (in [from, from + 2^width) of their places), n in
  // all, in order in the first CTA's list, from the entry that it returns on.
  __device__ __forceinline__ int gather(int b0, int b1, u64 from, int width, int n) {
    if (threadIdx.x == 0) sm.filled = 0;
    __syncthreads();
    members(b0, b1, from, width, [&](float, int, u64 p) {
      const int at = atomicAdd(&sm.filled, 1);
      if (at < kCap) sm.mine[at] = p;
    });
    sync();
    if (rank == 0) {
      int end[kMaxCluster];   // of each CTA's tokens in the list
#pragma unroll
      for (int j = 0; j < kMaxCluster; ++j) end[j] = cluster.map_shared_rank(&sm, j < ctas ? j : 0)->filled;
#pragma unroll
      for (int j = 0; j < kMaxCluster; ++j) end[j] = j < ctas ? end[j] : 0;
#pragma unroll
      for (int j = 1; j < kMaxCluster; ++j) end[j] += end[j - 1];
      for (int i = threadIdx.x; i < min(n, end[kMaxCluster - 1]); i += kThreads) {
        int j = 0, at = 0;
#pragma unroll
        for (int k = 0; k + 1 < kMaxCluster; ++k)
          if (i >= end[k]) {
            j = k + 1;
            at = end[k];
          }
        sm.place[i] = cluster.map_shared_rank(&sm, j)->mine[i - at];
      }
      __syncthreads();
    }
    if (ctas > 1) {   // (the others' lists are read; they go on)
      auto token = cluster.barrier_arrive();
      if (rank == 0) n = order(n);
      cluster.barrier_wait(std::move(token));
    } else {
      n = order(n);
    }
    return n;
  }
  // The list's n tokens in descending order of their places, with their weights.
  __device__ __forceinline__ int order(int n) {
    int at = 0;
    if (n <= kCount) {
      // by counting the larger ones
      const int i = threadIdx.x;
      if (i < n) {
        const u64 p = sm.place[i];
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) above += sm.place[j] > p;
        sm.place[kCount + above] = p;
      }
      at = kCount;
      __syncthreads();
    } else {
      // into 1024 parts of their range (of their logits, or indexes where those are equal), and by
      // counting the larger ones of a part
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
      uint32_t* start = sm.part_c;
      uint32_t* fill = sm.bins.cnt;
      uint32_t low = 0xffffffffu, top = 0;
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t k = (uint32_t)(sm.place[i] >> kSampleIndexBits);
        low = min(low, k);
        top = max(top, k);
      }
      low = __reduce_min_sync(0xffffffffu, low);
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) {
        sm.warp_c[warp] = low;
        sm.warp_i[warp] = top;
      }
      fill[2 * threadIdx.x] = fill[2 * threadIdx.x + 1] = 0;
      __syncthreads();
      low = __reduce_min_sync(0xffffffffu, sm.warp_c[lane % kWarps]);
      top = __reduce_max_sync(0xffffffffu, sm.warp_i[lane % kWarps]);
      const int width = top > low ? max(32 - __clz(top - low) - kDigit, 0) : kSampleIndexBits - kDigit;
      const auto part = [&](u64 p) {
        const uint32_t k = top > low ? (uint32_t)(p >> kSampleIndexBits) - low : (uint32_t)p & kIndexMask;
        return kBins - 1 - (int)(k >> width);
      };
      for (int i = threadIdx.x; i < n; i += kThreads) atomicAdd(&fill[part(sm.place[i])], 1u);
      __syncthreads();
      const uint32_t a = fill[2 * threadIdx.x], b = fill[2 * threadIdx.x + 1];
      if (__syncthreads_or(max(a, b) > kPart)) {
        // (many equal logits beside others: a call with 2000 of them behind one larger took 120 us, sorted 34)
        const int size = 1 << (32 - __clz(n - 1));
        for (int i = n + threadIdx.x; i < size; i += kThreads) sm.place[i] = 0;
        __syncthreads();
        sort_list(sm.place, size);
      } else {
        uint32_t run = a + b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, run, o);
          if (lane >= o) run += v;
        }
        if (lane == 31) sm.warp_i[warp] = run;
        __syncthreads();
        run -= a + b;
        for (int k = 0; k < warp; ++k) run += sm.warp_i[k];
        start[2 * threadIdx.x] = fill[2 * threadIdx.x] = run;
        start[2 * threadIdx.x + 1] = fill[2 * threadIdx.x + 1] = run + a;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads) {
          const u64 p = sm.place[i];
          sm.mine[atomicAdd(&fill[part(p)], 1u)] = p;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads) {
          const u64 p = sm.mine[i];
          const int b0 = start[part(p)], b1 = fill[part(p)];
          int above = b0;
          for (int j = b0; j < b1; ++j) above += sm.mine[j] > p;
          sm.place[above] = p;
        }
        __syncthreads();
      }
    }
    for (int i = threadIdx.x; i < n; i += kThreads) {
      float yh, yl;
      w.orders(logit_of(sm.place[at + i]), yh, yl);
      sm.weight[at + i] = weigh(token_of(sm.place[at + i]), yh, yl);
    }
    __syncthreads();
    return at;
  }

  // The end of the shortest run that holds `count` tokens, or weighs `mass` (count 0;
  // both within what there is): its place and its weight, in the first CTA's memory.
  // All CTAs of the cluster take part; the bins hold weights.
  __device__ __forceinline__ void find_run(uint32_t count, u64 mass) {
    for (int tries = 0; tries <= 2; ++tries) {   // (two windows hold everything)
      if (rank == 0) find_bin(sm.sum_w, sm.sum_c, sm.before_w, sm.before_c, count, mass, bin0);
      sync();
      const int to = first.bin;
      if (to >= 0) break;
      file<true>(to == kLower ? bin0 - kBins : bin0 + kBins);
    }
    const int bin = first.bin;
    int n = first.n, width = kPlaceBits;
    u64 from = 0;
    // more tokens than can be put in order: by their places in the bin's range, again by the parts'
    if (n > kCap) {
      const float2 y = bounds(bin, bin);
      // (a little more than the range on both sides)
      const float room = fabsf(w.max) * 0x1p-20f + y.x / w.ch * 0x1p-18f;
      const float top = w.max - y.x / w.ch + room, low = w.max - y.y / w.ch - room;
      if (top < kFinite && low > -kFinite) {   // (the last bin has no lower bound)
        from = place_of(low, (int)kIndexMask);
        width = 64 - __clzll((long long)(place_of(top, 0) - from));
      }
    }
    while (n > kCap && width > 0) {
      const int was = width;
      width = max(width - kDigit, 0);
      clear_bins(true);
      members(bin, bin, from, was, [&](float x, int i, u64 p) {
        float yh, yl;
        w.orders(x, yh, yl);
        const int b[1] = {kBins - 1 - (int)((p - from) >> width)};
        const u64 v[1] = {weigh(i, yh, yl)};
        add(b, v);
      });
      sum_bins<true>(sm.part_w, sm.part_c, &sm.base_w, &sm.base_c);
      if (rank == 0) {
        find_bin(sm.part_w, sm.part_c, sm.base_w, sm.base_c, count, mass, 0);
        if (threadIdx.x == 0) sm.from = from + ((u64)(kBins - 1 - sm.bin) << width);
      }
      sync();
      n = first.n;
      from = first.from;
    }
    n = min(n, kCap);   // (places are all different)
    const int at = gather(bin, bin, from, width, n);
    if (rank == 0) {
      Scan<kThreads> sc{sm, at, n};
      u64 weight;
      int i;
      if (count) {
        i = (int)(count - sm.base_c) - 1;
        sc.n = i + 1;
        sc.sum();
        weight = sc.total();
      } else {
        sc.sum();
        i = sc.reach(mass - sm.base_w, weight);
      }
      if (threadIdx.x == 0) {
        sm.run_place = sm.place[at + i];
        sm.run_w = sm.base_w + weight;
      }
    }
    sync();
  }
};

// What a row wants of its distribution.
struct Wanted {
  int top_k;
  float top_p, u, u_next;
  bool last;      // no draft follows: draw
};

// Whether a draft of weight (s + r) 2^-n, or none, stays.
__device__ __forceinline__ bool draft_stays(const Smem& sm, const Row& w, float x, int draft, bool kept, u64 total,
                                            float u) {
  if (!kept) return false;
  float yh, yl, s, r;
  int n;
  w.orders(x, yh, yl);
  if (!(yh < 1024.f)) return false;
  pow2_neg(sm.pow2, yh, yl, s, r, n);
  const double q = w.q ? (double)w.q[draft] : 1.;
  // u q < w / total
  return (double)u * q * ((double)total * 0x1p-44) < scalbn((double)s + (double)r, -n);
}

// The rest of a row whose kept tokens are among the n of the first CTA's list, by
// one warp or the CTA: what is kept, and the token.  -1: the draft stays.
template <int THREADS, class T>
__device__ __forceinline__ u64 decide(Sampler<T>& s, const Wanted& want, int at, int n, u64& total, u64& kept,
                                      bool& stays) {
  Smem& sm = s.sm;
  if (want.top_k > 0) n = min(n, want.top_k);
  Scan<THREADS> sc{sm, at, n};
  sc.sum();
  if (want.top_k > 0) total = sc.total();
  if (want.top_p < 1.f) {
    u64 weight;
    sc.n = n = sc.reach(max(share(total, want.top_p, true), 1ull), weight) + 1;
    total = weight;
  }
  kept = sm.place[at + n - 1];
  stays = false;
  if (!want.last) {
    if (threadIdx.x == 0) {
      const int d = s.w.draft;
      const float x = s.w.draft_x;
      sm.stays = draft_stays(sm, s.w, x, d, s.w.draft_in && x >= s.w.floor && place_of(x, d) >= kept, total, want.u);
    }
    Scan<THREADS>::sync();
    stays = sm.stays != 0;
    if (stays) return 0;
    // what the draft left of the kept tokens, if anything
    s.w.rest = true;
    s.w.set_total(total);
    u64 mine[kPer], some = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = sc.entry(k);
      mine[k] = i < n ? s.left(sm.weight[at + i], token_of(sm.place[at + i])) : 0;
      some |= mine[k];
    }
    if (THREADS == 32 ? __any_sync(0xffffffffu, some != 0) : __syncthreads_or(some != 0)) {
      Scan<THREADS>::sync();
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (sc.entry(k) < n) sm.weight[at + sc.entry(k)] = mine[k];
      Scan<THREADS>::sync();
      sc.sum();
      total = sc.total();
    }
  }
  u64 weight;
  return sm.place[at + sc.reach(share(total, want.u_next, false), weight)];
}

template <class T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int r = blockIdx.x / ctas;   // row
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  dev::pdl_trigger();
  for (int i = threadIdx.x; i < 1024; i += kThreads) sm.pow2[i] = make_float2(kPow2.hi[i], kPow2.lo[i]);
  dev::pdl_wait();

  // the row's request, and the draft after it (-1: none, the sequence's last row)
  int req = r, draft = -1;
  Wanted want;
  want.last = true;
  if (p.cu) {
    int a = 0, b = p.n_seq + 1;       // first entry above r
    while (a < b) {
      const int m = (a + b) >> 1;
      if (p.cu[m] <= r) a = m + 1;
      else b = m;
    }
    req = a - 1;
    if (req < 0 || req >= p.n_seq) return;   // (the whole cluster)
    want.last = r + 1 >= min(p.cu[req + 1], p.rows);
    if (!want.last) draft = p.tokens[r + 1];
  }
  // (every CTA of the cluster runs before its memory is written: waited for below)
  auto arrived = cluster.barrier_arrive();
  float heat = p.s.temperature ? p.s.temperature[req] : 1.f;
  want.top_k = p.s.top_k ? p.s.top_k[req] : 0;
  const float min_p = p.s.min_p ? p.s.min_p[req] : 0.f;
  want.top_p = p.s.top_p ? p.s.top_p[req] : 1.f;
  want.u = p.cu && want.last ? 0.f : p.u[r];
  want.u_next = p.cu ? p.u_next[req] : want.u;
  const T* row = static_cast<const T*>(p.logits) + p.stride * r;
  const int per = (p.vocab + ctas - 1) / ctas;
  const int lo = min(rank * per, p.vocab), hi = min(lo + per, p.vocab);

  // the largest logit (NaN if there is one)
  float best = -INFINITY;
  for_tokens<4>(row, lo, hi, [&](const float (&x)[4], int i, int n) {
    best = max_nan(best, x[0]);
    if (n > 1) best = max_nan(max_nan(best, x[1]), max_nan(x[2], x[3]));
  });
  bool bad = best != best || !(heat == 0.f || (heat >= 0x1p-64f && heat <= 0x1p64f)) || min_p != min_p ||
             want.top_p != want.top_p || !(want.u >= 0.f && want.u < 1.f) || !(want.u_next >= 0.f && want.u_next < 1.f);
  if (heat == 0.f) {
    heat = 1.f;
    want.top_k = 1;
  }
  if (warp == 1 && lane == 0 && min_p > 0.f) sm.min_orders = (double)heat * log((double)fminf(min_p, 1.f));
  // (a row without a distribution: no key is that large)
  uint32_t key = bad ? 0xffffffffu : (uint32_t)(place_of(best, 0) >> kSampleIndexBits);
  key = __reduce_max_sync(0xffffffffu, key);
  if (lane == 0) sm.warp_c[warp] = key;
  __syncthreads();
  key = __reduce_max_sync(0xffffffffu, sm.warp_c[lane % kWarps]);
  cluster.barrier_wait(std::move(arrived));
  if (threadIdx.x < ctas) {
    Smem* o = cluster.map_shared_rank(&sm, threadIdx.x);
    o->best_key[rank] = key;
  }
  if (ctas > 1) cluster.sync();
  else __syncthreads();
  key = __reduce_max_sync(0xffffffffu, lane < ctas ? sm.best_key[lane] : 0);
  best = logit_of((u64)key << kSampleIndexBits);
  bad = key == 0xffffffffu || best == -INFINITY;
  float* dist = p.dist ? p.dist + p.dist_stride * r : nullptr;
  // (of what follows every CTA of the cluster decides alike)
  const bool certain = want.top_k == 1 || want.top_p <= 0.f;   // only the first token is kept
  int top_token = 0;
  if (certain && !bad) {
    uint32_t at = kIndexMask;
    for_tokens<4>(row, lo, hi, [&](const float (&x)[4], int i, int n) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (x[k] == best) at = min(at, (uint32_t)(i + k));
    });
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) sm.warp_i[warp] = at;
    __syncthreads();
    at = __reduce_min_sync(0xffffffffu, sm.warp_i[lane % kWarps]);
    if (threadIdx.x < ctas) cluster.map_shared_rank(&sm, threadIdx.x)->best_i[rank] = at;
    if (ctas > 1) cluster.sync();
    else __syncthreads();
    top_token = (int)__reduce_min_sync(0xffffffffu, lane < ctas ? sm.best_i[lane] : kIndexMask);
  }
  if (bad || (certain && !p.cu)) {
    if (dist)
      for (int i = lo + threadIdx.x; i < hi; i += kThreads) dist[i] = !bad && i == top_token ? 1.f : 0.f;
    if (rank == 0 && threadIdx.x == 0) {
      if (p.cu) {
        p.outcome[r] = -1;
      } else {
        p.token[r] = bad ? -1 : top_token;
        if (p.prob) p.prob[r] = bad ? 0.f : 1.f;
      }
    }
    return;
  }

  Sampler<T> s{sm, *cluster.map_shared_rank(&sm, 0), cluster, row, lo, hi, rank, ctas};
  s.w.max = fminf(best, kFinite);
  {
    constexpr float kLog2eH = 1.44269502162933349609375f, kLog2eL = 1.92596299112661746887e-08f;
    s.w.ch = kLog2eH / heat;
    s.w.cl = (fmaf(-s.w.ch, heat, kLog2eH) + kLog2eL) / heat;
  }
  s.w.floor = best == INFINITY ? INFINITY
              : min_p > 0.f    ? __double2float_ru((double)best + sm.min_orders)
                               : -INFINITY;
  s.w.rest = false;
  s.w.kept = 0;
  u64 kept = 0, total = 1ull << kFix;
  s.w.q = p.q ? p.q + p.q_stride * r : nullptr;
  s.w.draft = draft;
  s.w.draft_in = draft >= 0 && draft < p.vocab;
  s.w.draft_x = s.w.draft_in ? to_float(row[draft]) : 0.f;
  s.w.set_total(total);

  bool listed = certain;            // the kept tokens are in the first CTA's list, in order
  int at = 0, n = 1;
  if (certain) {
    if (threadIdx.x == 0) {
      sm.place[0] = place_of(best, top_token);
      sm.weight[0] = total;
    }
    __syncthreads();
  } else {
    if (want.top_k > 0) s.template file<false>(0);
    else s.template file<true>(0);
    // few tokens up to the end of the kept ones: they are all that the rest needs
    if (rank == 0 && (want.top_k > 0 || want.top_p < 1.f))
      s.find_bin(sm.sum_w, sm.sum_c, sm.before_w, sm.before_c,
                 want.top_k > 0 ? min((uint32_t)want.top_k, sm.total_c) : 0,
                 want.top_k > 0 ? 0 : share(sm.total_w, want.top_p, true), 0);
    s.sync();
    const uint32_t tokens = s.first.total_c;
    total = s.first.total_w;
    if (want.top_k > 0 || want.top_p < 1.f) {
      const int bin = s.first.bin;
      n = bin >= 0 ? s.first.base_c + s.first.n : kCap + 1;
      listed = n <= kCap;
      if (listed) {
        at = s.gather(0, bin, 0, kPlaceBits, n);
      } else {
        s.sync();   // (the first CTA's memory has been read)
        if (want.top_k > 0) {
          s.template file<true>(0);
          s.sync();
          total = s.first.total_w;
        }
        if (want.top_k > 0 && (uint32_t)want.top_k < tokens) {
          s.find_run(want.top_k, 0);
          kept = s.first.run_place;
          total = s.first.run_w;
        }
        if (want.top_p < 1.f) {
          s.find_run(0, share(total, want.top_p, true));
          kept = s.first.run_place;
          total = s.first.run_w;
        }
      }
    }
  }
  bool stays = false;
  u64 place = 0;
  if (listed) {
    if (rank && !dist) return;   // (the first CTA has what it needs)
    if (rank == 0) {
      if (n <= 32 * kPer) {
        if (warp == 0) place = decide<32>(s, want, at, n, total, kept, stays);
      } else {
        place = decide<kThreads>(s, want, at, n, total, kept, stays);
      }
    }
    if (dist) {   // (no drafts then: the row's own distribution)
      if (rank == 0 && threadIdx.x == 0) {
        sm.kept = kept;
        sm.kept_w = total;
      }
      s.sync();
      kept = s.first.kept;
      total = s.first.kept_w;
    }
  } else {
    if (!want.last) {
      // does the draft stay?
      if (threadIdx.x == 0)
        sm.stays = draft_stays(sm, s.w, s.w.draft_x, draft,
                               s.w.draft_in && s.w.draft_x >= s.w.floor && place_of(s.w.draft_x, draft) >= kept, total,
                               want.u);
      __syncthreads();
      stays = sm.stays != 0;   // (every CTA finds the same)
      if (!stays) {
        s.sync();
        s.w.rest = true;
        s.w.kept = kept;
        s.w.set_total(total);
        s.template file<true>(0);
        s.sync();
        const u64 left = s.first.total_w;
        if (left) {
          total = left;
        } else {
          s.sync();         // (everyone has read it)
          s.w.rest = false;
          s.template file<true>(0);
          s.sync();
        }
      }
    }
    if (!stays) {
      s.find_run(0, share(total, want.u_next, false));
      place = s.first.run_place;
    }
  }
  if (rank == 0 && threadIdx.x == 0) {
    const int token = token_of(place);
    if (p.cu) {
      p.outcome[r] = stays ? kStays : token;
    } else {
      p.token[r] = token;
      if (p.prob) {
        float yh, yl, a, b;
        int m;
        s.w.orders(logit_of(place), yh, yl);
        pow2_neg(sm.pow2, yh, yl, a, b, m);
        p.prob[r] = share_of(a, b, m, pair_of(total));
      }
    }
  }
  if (dist) {
    const float2 sum = pair_of(total);
    const float ih = 1.f / sum.x, il = (fmaf(-ih, sum.x, 1.f) - ih * sum.y) * ih;
    for_tokens<1>(row, lo, hi, [&](const float (&x)[4], int i, int n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v = 0.f, yh, yl;
        s.w.orders(x[k], yh, yl);
        if (x[k] >= s.w.floor && yh < 152.f && place_of(x[k], i + k) >= kept) {
          float a, b;
          int m;
          pow2_neg(sm.pow2, yh, yl, a, b, m);
          const float h = a * ih;
          v = h + (fmaf(a, ih, -h) + fmaf(a, il, b * ih));
          // (in two steps, of which only the second may leave the normal numbers)
          const int q = min(m, 100);
          v = v * __int_as_float((127 - q) << 23) * __int_as_float((127 - (m - q)) << 23);
        }
        if (k < n) dist[i + k] = v;
      }
    });
  }
  if (ctas > 1 && (!listed || dist)) cluster.sync();   // (the first CTA's memory is read to the end)
}

// One warp per sequence: the first row whose draft does not stay.
__global__ void __launch_bounds__(256) accept_kernel(const SampleParams p) {
  dev::pdl_trigger();
  dev::pdl_wait();
  const int b = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= p.n_seq) return;
  const int r0 = max(p.cu[b], 0), r1 = min(p.cu[b + 1], p.rows);
  int at = r0, token = -1;
  for (; at < r1; at += 32) {
    const int v = at + lane < r1 ? p.outcome[at + lane] : kStays;
    const uint32_t stop = __ballot_sync(0xffffffffu, v != kStays);
    if (stop) {
      const int k = __ffs(stop) - 1;
      at += k;
      token = __shfl_sync(0xffffffffu, v, k);
      break;
    }
  }
  if (lane == 0) {
    p.accepted[b] = r1 > r0 ? min(at, r1 - 1) - r0 : 0;
    p.next[b] = token;
  }
}

template <class T>
cudaError_t launch(const SampleParams& p, int ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.rows * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)ctas, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
}

}  // namespace

cudaError_t sample_setup() {
  void (*ks[3])(SampleParams) = {sample_kernel<float>, sample_kernel<__nv_bfloat16>, sample_kernel<__half>};
  for (auto k : ks) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_sample(const SampleParams& p, int sms, cudaStream_t st) {
  // CTAs of a row: up to 8/3 on each SM (two run at a time, and rows are over at different times), with 2048
  // tokens each at least.  More cost more to clear, sum and wait for than they share.  With 1, 2, 4, 8 a row,
  // in us: 64 rows of 32000 49, 40, 33, 50; 100 of 128000 161, 122, 105, 131; 160 of 128000 216, 143,
  // 156, 197; 300 of 32000 71, 81, 103, 167.
  int ctas = 1;
  while (ctas < kMaxCluster && 3ll * p.rows * ctas <= 4 * sms && p.vocab >= 4096 * ctas) ctas *= 2;
  cudaError_t e = p.rows == 0             ? cudaSuccess
                  : p.type == KVR_ACT_F32 ? launch<float>(p, ctas, st)
                  : p.type == KVR_ACT_BF16 ? launch<__nv_bfloat16>(p, ctas, st)
                                           : launch<__half>(p, ctas, st);
  if (e != cudaSuccess || !p.cu) return e;
  return launch_k(accept_kernel, dim3((p.n_seq + 7) / 8), dim3(256), 0, st, p);
}

}  // namespace kvr
