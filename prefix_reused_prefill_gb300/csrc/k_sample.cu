// Sampling from given random numbers, and speculative sampling (include/kvr.h).
//
// A row's tokens are never sorted.  Everything asked of their order is of one kind:
// the shortest run from the largest logit that holds a count (top_k) or a weight
// (top_p; the drawn token ends the run that holds more than u of the weight).  So
// one pass files every token under its logit's distance from the maximum, in bins
// of 1/32 of a binary order that hold the count and the weight; running sums over
// the bins name the bin in which a run ends, and only that bin's tokens are put in
// order.
//
// A token's place is one 50-bit number, its logit's bits above its inverted
// index, so equal logits need no care.  Weights are formed to 2^-46 in pairs
// of floats and summed as whole numbers of 2^-44 of the largest: whole numbers have
// one sum in any order, so shared-memory atomics serve and every pass, CTA and
// launch agrees on where a run ends.
#include <cooperative_groups.h>

#include "kvr_batch.cuh"

namespace cg = cooperative_groups;

namespace kvr {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1536;
constexpr float kBinScale = 32.f;
constexpr float kOrders = kBins / kBinScale;   // what is further from the maximum weighs nothing (last bin)
constexpr int kCopies = 4;           // of the bins, by lane: equal logits are neighbours in a bin
constexpr int kFix = 44;
constexpr int kCap = 2048;           // tokens that one CTA puts in order
constexpr int kDigit = 10;           // bits of a place taken at a time where a bin holds more
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
  uint32_t cnt[kCopies][kBins], lo[kCopies][kBins], hi[kCopies][kBins];
};
struct Smem {
  float2 pow2[1024];
  Bins bins;
  // of the cluster's first CTA: running weights and counts over the row's bins, over the parts of one bin,
  // and the tokens of one bin
  u64 sum_w[kBins], part_w[kBins];
  uint32_t sum_c[kBins], part_c[kBins];
  u64 place[kCap], weight[kCap];
  u64 warp_w[kWarps];
  uint32_t warp_c[kWarps];
  // what the CTAs tell one another
  float max_[kMaxCluster];
  int bad_[kMaxCluster];
  int n, bin;             // tokens of the bin in which a run ends
  u64 base_w;             // weight and count before it
  uint32_t base_c;
  u64 from;               // first place of a part of it
  u64 run_place, run_w;   // the end of a run, its weight and that of its last token
  u64 last_w;
  int fill;
  int stays;
};

// What a row's tokens weigh.
struct Row {
  float max;
  float ch, cl;         // log2(e) / temperature
  float floor;          // logits below weigh less than min_p
  // of a rejected draft's row: weight beyond the drafter's
  const float* q;       // null: all weight of `draft` goes
  double total;
  int draft;
  u64 kept;             // places from here on
  bool rest;

  // binary orders below the maximum, as a pair; false where a token weighs nothing
  __device__ __forceinline__ bool orders(float x, float& yh, float& yl) const {
    if (x == max) {     // (also at infinity)
      yh = yl = 0.f;
      return true;
    }
    const float d = max - x;
    const float b = d - max;
    const float dl = (max - (d - b)) - (x + b);
    yh = d * ch;
    yl = fmaf(d, ch, -yh) + fmaf(d, cl, dl * ch);
    return yh < kOrders;
  }
};

__device__ __forceinline__ u64 place_of(float x, int i) {
  const uint32_t b = __float_as_uint(x + 0.f);   // (-0 is 0)
  const uint32_t k = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  return ((u64)k << kSampleIndexBits) | (kIndexMask - (uint32_t)i);
}

// 2^-(yh + yl) = (s + r) 2^-n: the nearest of 1024 steps from the table, the
// rest by its series, whose first term is a pair of floats.
__device__ __forceinline__ void pow2_neg(const float2* tab, float yh, float yl, float& s, float& r, int& n) {
  constexpr float kLn2h = 0.693147182464599609375f;
  constexpr float kLn2l = -1.904654323148236e-09f;
  const int j = __float2int_rn(yh * 1024.f);
  const float f = fmaf((float)j, -1.f / 1024.f, yh);
  const float zh = -f * kLn2h;
  const float zl = fmaf(-f, kLn2h, -zh) - fmaf(f, kLn2l, yl * kLn2h);
  const float e = fmaf(zh * zh, fmaf(zh, 1.f / 6.f, 0.5f), zl);
  const float2 t = tab[j & 1023];
  n = j >> 10;
  const float a = t.x * zh;
  float al = fmaf(t.x, zh, -a);
  al = fmaf(t.y, zh, al) + fmaf(t.x, e, t.y);
  s = t.x + a;
  r = (a - (s - t.x)) + al;
}

__device__ __forceinline__ u64 weight_fixed(const float2* tab, float yh, float yl) {
  float s, r;
  int n;
  pow2_neg(tab, yh, yl, s, r, n);
  const float scale = __int_as_float((kFix - n + 127) << 23);
  return (u64)(__float2ll_rn(s * scale) + (long long)__float2int_rn(r * scale));
}

__device__ __forceinline__ int bin_of(float yh) { return min((int)(yh * kBinScale), kBins - 1); }

// f(logit, token) over the CTA's part [lo, hi) of a row: 16-byte loads but at the ends.
template <class T, class F>
__device__ __forceinline__ void for_tokens(const T* row, int lo, int hi, F f) {
  constexpr int kV = 16 / sizeof(T);
  const int skip = (int)((16 - ((uintptr_t)(row + lo) & 15)) & 15) / (int)sizeof(T);
  const int a = min(lo + skip, hi), b = a + (hi - a) / kV * kV;
  for (int i = lo + threadIdx.x; i < a; i += kThreads) f(to_float(row[i]), i);
  for (int i = a + threadIdx.x * kV; i < b; i += kThreads * kV) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + i);
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int k = 0; k < kV; ++k) f(to_float(e[k]), i + k);
  }
  for (int i = b + threadIdx.x; i < hi; i += kThreads) f(to_float(row[i]), i);
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

template <class T>
struct Sampler {
  Smem& sm;
  Smem& first;          // the cluster's first CTA's
  const cg::cluster_group& cluster;
  const T* row;
  int lo, hi;           // this CTA's tokens
  int rank;
  Row w;

  __device__ __forceinline__ void clear_bins() {
    uint32_t* b = reinterpret_cast<uint32_t*>(&sm.bins);
    for (int i = threadIdx.x; i < (int)(sizeof(Bins) / 4); i += kThreads) b[i] = 0;
    __syncthreads();
  }
  __device__ __forceinline__ void add(int bin, u64 v) {
    const int c = threadIdx.x % kCopies;
    atomicAdd(&sm.bins.cnt[c][bin], 1u);
    const uint32_t l = (uint32_t)v, h = (uint32_t)(v >> 32);
    if (l) {
      const uint32_t old = atomicAdd(&sm.bins.lo[c][bin], l);
      const uint32_t carry = old + l < old ? 1u : 0u;
      if (h + carry) atomicAdd(&sm.bins.hi[c][bin], h + carry);
    } else if (h) {
      atomicAdd(&sm.bins.hi[c][bin], h);
    }
  }

  // Running sums over the cluster's bins, to the first CTA's sum_w and sum_c.
  __device__ __forceinline__ void sum_bins(u64* sum_w, uint32_t* sum_c) {
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kThreads) {
      uint32_t c = 0, l = 0, h = 0;
#pragma unroll
      for (int k = 0; k < kCopies; ++k) {
        c += sm.bins.cnt[k][b];
        const uint32_t o = l;
        l += sm.bins.lo[k][b];
        h += sm.bins.hi[k][b] + (l < o ? 1u : 0u);
      }
      sm.bins.cnt[0][b] = c;
      sm.bins.lo[0][b] = l;
      sm.bins.hi[0][b] = h;
    }
    cluster.sync();
    if (rank == 0) {
      constexpr int kPer = kBins / kThreads;
      u64 v[kPer];
      uint32_t c[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int b = threadIdx.x * kPer + k;
        v[k] = 0;
        c[k] = 0;
        for (int j = 0; j < (int)cluster.num_blocks(); ++j) {
          const Bins& o = cluster.map_shared_rank(&sm, j)->bins;
          v[k] += (u64)o.hi[0][b] << 32 | o.lo[0][b];
          c[k] += o.cnt[0][b];
        }
        if (k) {
          v[k] += v[k - 1];
          c[k] += c[k - 1];
        }
      }
      u64 bv;
      uint32_t bc;
      block_before(v[kPer - 1], c[kPer - 1], bv, bc);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        sum_w[threadIdx.x * kPer + k] = bv + v[k];
        sum_c[threadIdx.x * kPer + k] = bc + c[k];
      }
      __syncthreads();
    }
  }

  // sums of the threads in front
  __device__ __forceinline__ void block_before(u64 v, uint32_t c, u64& bv, uint32_t& bc) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 rv = v;
    uint32_t rc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 a = __shfl_up_sync(0xffffffffu, rv, o);
      const uint32_t b = __shfl_up_sync(0xffffffffu, rc, o);
      if (lane >= o) {
        rv += a;
        rc += b;
      }
    }
    __syncthreads();
    if (lane == 31) {
      sm.warp_w[warp] = rv;
      sm.warp_c[warp] = rc;
    }
    __syncthreads();
    bv = rv - v;
    bc = rc - c;
    for (int k = 0; k < warp; ++k) {
      bv += sm.warp_w[k];
      bc += sm.warp_c[k];
    }
  }

  // The bin in which the run that holds `count` tokens or (count 0) `mass` ends, by
  // the bins' running sums and what stands in front of them.  First CTA only.
  __device__ __forceinline__ void find_bin(const u64* sum_w, const uint32_t* sum_c, uint32_t count, u64 mass,
                                           u64 before_w, uint32_t before_c) {
    for (int b = threadIdx.x; b < kBins; b += kThreads) {
      const u64 iw = before_w + sum_w[b], pw = before_w + (b ? sum_w[b - 1] : 0);
      const uint32_t ic = before_c + sum_c[b], pc = before_c + (b ? sum_c[b - 1] : 0);
      if (count ? ic >= count && pc < count : iw >= mass && pw < mass) {
        sm.bin = b;
        sm.n = (int)(ic - pc);
        sm.base_w = pw;
        sm.base_c = pc;
      }
    }
    __syncthreads();
  }

  // n tokens (place, weight) of the first CTA's list, in descending order of their places
  __device__ __forceinline__ void order(int n) {
    int size = 2;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += kThreads) {
      sm.place[i] = 0;
      sm.weight[i] = 0;
    }
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1)
      for (int j = k >> 1; j > 0; j >>= 1) {
        for (int t = threadIdx.x; t < size / 2; t += kThreads) {
          const int i = 2 * j * (t / j) + t % j;
          const u64 a = sm.place[i], b = sm.place[i + j];
          if ((a < b) == ((i & k) == 0)) {
            sm.place[i] = b;
            sm.place[i + j] = a;
            const u64 x = sm.weight[i];
            sm.weight[i] = sm.weight[i + j];
            sm.weight[i + j] = x;
          }
        }
        __syncthreads();
      }
  }

  // Whether a token belongs to a bin (and, where the row's weight is what a draft
  // left, is kept); its distance from the maximum.
  __device__ __forceinline__ bool member(float x, int i, int bin, float& yh, float& yl) const {
    if (!(x >= w.floor)) return false;
    const bool some = w.orders(x, yh, yl);
    if ((some ? bin_of(yh) : kBins - 1) != bin) return false;
    return !w.rest || (some && place_of(x, i) >= w.kept);
  }
  __device__ __forceinline__ u64 weigh(float x, int i, float yh, float yl) const {
    if (!(yh < kOrders)) return 0;
    const u64 v = weight_fixed(sm.pow2, yh, yl);
    if (!w.rest) return v;
    if (!w.q) return i == w.draft ? 0 : v;
    const double left = (double)v - (double)w.q[i] * w.total;
    return left > 0. ? (u64)__double2ll_rn(left) : 0;
  }

  // The row's tokens into the bins, and the bins' running sums.  With `rest`
  // only what weighs: tokens that a draft's row no longer has are none.
  __device__ __forceinline__ void file() {
    clear_bins();
    uint32_t behind = 0;
    for_tokens(row, lo, hi, [&](float x, int i) {
      if (!(x >= w.floor)) return;
      float yh, yl;
      if (!w.orders(x, yh, yl)) {
        ++behind;
        return;
      }
      if (w.rest && place_of(x, i) < w.kept) return;
      add(bin_of(yh), weigh(x, i, yh, yl));
    });
    behind = w.rest ? 0 : __reduce_add_sync(0xffffffffu, behind);
    if ((threadIdx.x & 31) == 0 && behind) atomicAdd(&sm.bins.cnt[0][kBins - 1], behind);
    sum_bins(sm.sum_w, sm.sum_c);
    cluster.sync();
  }

  // The end of the shortest run that holds `count` tokens, or weighs `mass` (count 0;
  // both within what there is): its place, its weight, its last token's weight.
  // All CTAs of the cluster take part; the results are in the first one's memory.
  __device__ __forceinline__ void find_run(uint32_t count, u64 mass) {
    if (rank == 0) {
      find_bin(sm.sum_w, sm.sum_c, count, mass, 0, 0);
      if (threadIdx.x == 0) sm.fill = 0;
    }
    cluster.sync();
    const int bin = first.bin;
    int n = first.n, shift = kPlaceBits;
    u64 from = 0;
    // more tokens than can be put in order: by the next bits of their places
    while (n > kCap) {
      shift -= kDigit;
      clear_bins();
      for_tokens(row, lo, hi, [&](float x, int i) {
        float yh, yl;
        if (!member(x, i, bin, yh, yl)) return;
        const u64 p = place_of(x, i);
        if (p < from || (p - from) >> (shift + kDigit)) return;
        add((1 << kDigit) - 1 - (int)((p - from) >> shift), weigh(x, i, yh, yl));
      });
      sum_bins(sm.part_w, sm.part_c);
      if (rank == 0) {
        find_bin(sm.part_w, sm.part_c, count, mass, sm.base_w, sm.base_c);
        if (threadIdx.x == 0) sm.from = from + ((u64)((1 << kDigit) - 1 - sm.bin) << shift);
      }
      cluster.sync();
      n = first.n;
      from = first.from;
    }
    for_tokens(row, lo, hi, [&](float x, int i) {
      float yh, yl;
      if (!member(x, i, bin, yh, yl)) return;
      const u64 p = place_of(x, i);
      if (p < from || (p - from) >> shift) return;
      const int at = atomicAdd(&first.fill, 1);
      if (at < kCap) {
        first.place[at] = p;
        first.weight[at] = weigh(x, i, yh, yl);
      }
    });
    cluster.sync();
    if (rank == 0) {
      order(n);
      constexpr int kPer = kCap / kThreads;
      u64 v[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int i = threadIdx.x * kPer + k;
        v[k] = (i < n ? sm.weight[i] : 0) + (k ? v[k - 1] : 0);
      }
      u64 bv;
      uint32_t bc;
      block_before(v[kPer - 1], 0, bv, bc);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int i = threadIdx.x * kPer + k;
        const u64 iw = sm.base_w + bv + v[k], pw = sm.base_w + bv + (k ? v[k - 1] : 0);
        if (i < n && (count ? sm.base_c + i + 1 == count : iw >= mass && pw < mass)) {
          sm.run_place = sm.place[i];
          sm.run_w = iw;
        }
      }
    }
    cluster.sync();
  }
};

// exp((x - max) / temperature) / total of one token, in 64 bits
__device__ double share_of(double x, double max, double heat, u64 total) {
  const double w = x == max ? 1. : exp((x - max) / heat);
  return w / ((double)total * (1. / (double)(1ull << kFix)));
}

template <class T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int r = blockIdx.x / ctas;   // row
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  // the row's request, and the draft after it (-1: none, the sequence's last row)
  int req = r, draft = -1;
  bool last = true;
  if (p.cu) {
    int a = 0, b = p.n_seq + 1;       // first entry above r
    while (a < b) {
      const int m = (a + b) >> 1;
      if (p.cu[m] <= r) a = m + 1;
      else b = m;
    }
    req = a - 1;
    if (req < 0 || req >= p.n_seq) return;   // (the whole cluster)
    last = r + 1 >= min(p.cu[req + 1], p.rows);
    if (!last) draft = p.tokens[r + 1];
  }
  float heat = p.s.temperature ? p.s.temperature[req] : 1.f;
  int top_k = p.s.top_k ? p.s.top_k[req] : 0;
  const float min_p = p.s.min_p ? p.s.min_p[req] : 0.f;
  const float top_p = p.s.top_p ? p.s.top_p[req] : 1.f;
  const float u = !p.cu ? p.u[r] : last ? 0.f : p.u[r];
  const float u_next = p.cu ? p.u_next[req] : u;
  bool bad = !(heat == 0.f || (heat >= 0x1p-64f && heat <= 0x1p64f)) || min_p != min_p || top_p != top_p ||
             !(u >= 0.f && u < 1.f) || !(u_next >= 0.f && u_next < 1.f);
  if (heat == 0.f) {
    heat = 1.f;
    top_k = 1;
  }

  cluster.sync();   // every CTA of the cluster runs: its memory may be written
  for (int i = threadIdx.x; i < 1024; i += kThreads) sm.pow2[i] = make_float2(kPow2.hi[i], kPow2.lo[i]);

  const T* row = static_cast<const T*>(p.logits) + p.stride * r;
  const int per = (p.vocab + ctas - 1) / ctas;
  const int lo = min(rank * per, p.vocab), hi = min(lo + per, p.vocab);

  // the largest logit
  float best = -INFINITY;
  bool nan = false;
  for_tokens(row, lo, hi, [&](float x, int) {
    best = fmaxf(best, x);
    nan |= x != x;
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  float* red = reinterpret_cast<float*>(sm.warp_w);
  if (lane == 0) red[warp] = best;
  nan = __syncthreads_or(nan);
  if (threadIdx.x == 0) {
    for (int k = 1; k < kWarps; ++k) best = fmaxf(best, red[k]);
    for (int j = 0; j < ctas; ++j) {
      Smem* o = cluster.map_shared_rank(&sm, j);
      o->max_[rank] = best;
      o->bad_[rank] = nan;
    }
  }
  cluster.sync();
  best = sm.max_[0];
  bad |= sm.bad_[0] != 0;
  for (int j = 1; j < ctas; ++j) {
    best = fmaxf(best, sm.max_[j]);
    bad |= sm.bad_[j] != 0;
  }
  bad |= best == -INFINITY;
  float* dist = p.dist ? p.dist + p.dist_stride * r : nullptr;
  if (bad) {   // (every CTA of the cluster alike)
    if (dist)
      for (int i = lo + threadIdx.x; i < hi; i += kThreads) dist[i] = 0.f;
    if (rank == 0 && threadIdx.x == 0) {
      if (p.cu) {
        p.outcome[r] = -1;
      } else {
        p.token[r] = -1;
        if (p.prob) p.prob[r] = 0.f;
      }
    }
    return;
  }

  const double c = 1.4426950408889634074 / (double)heat;
  Row w;
  w.max = best;
  w.ch = (float)c;
  w.cl = (float)(c - (double)w.ch);
  w.floor = min_p > 0.f ? __double2float_ru((double)best + (double)heat * log((double)fminf(min_p, 1.f))) : -INFINITY;
  w.rest = false;
  w.kept = 0;
  w.q = p.q ? p.q + p.q_stride * r : nullptr;
  w.draft = draft;
  w.total = 0.;
  Sampler<T> s{sm, *cluster.map_shared_rank(&sm, 0), cluster, row, lo, hi, rank, w};
  s.file();
  u64 total = s.first.sum_w[kBins - 1];
  const uint32_t tokens = s.first.sum_c[kBins - 1];
  u64 kept = 0;
  if (top_k > 0 && (uint32_t)top_k < tokens) {
    s.find_run(top_k, 0);
    kept = s.first.run_place;
    total = s.first.run_w;
  }
  if (top_p < 1.f) {
    const u64 t = top_p > 0.f ? share(total, top_p, true) : 1;
    s.find_run(0, t);
    kept = s.first.run_place;
    total = s.first.run_w;
  }

  if (p.cu && !last) {
    // does the draft stay?
    if (rank == 0 && threadIdx.x == 0) {
      double pd = 0.;
      if (draft >= 0 && draft < p.vocab) {
        const float x = to_float(row[draft]);
        if (x >= w.floor && place_of(x, draft) >= kept) pd = share_of(x, best, heat, total);
      }
      const double qd = !s.w.q ? 1. : draft >= 0 && draft < p.vocab ? (double)s.w.q[draft] : 1.;
      sm.stays = (double)u * qd < pd;
      if (sm.stays) p.outcome[r] = kStays;
    }
    cluster.sync();
    const bool stays = s.first.stays != 0;
    if (!stays) {
      s.w.rest = true;
      s.w.kept = kept;
      s.w.total = (double)total;
      s.file();
      const u64 left = s.first.sum_w[kBins - 1];
      if (left) {
        total = left;
      } else {
        cluster.sync();   // (everyone has read it)
        s.w.rest = false;
        s.file();
      }
    }
    if (stays) {
      cluster.sync();     // (the first CTA's memory has been read)
      return;
    }
  }
  s.find_run(0, share(total, u_next, false));
  const u64 place = s.first.run_place;
  if (rank == 0 && threadIdx.x == 0) {
    const int token = (int)(kIndexMask - (uint32_t)(place & kIndexMask));
    if (p.cu) {
      p.outcome[r] = token;
    } else {
      p.token[r] = token;
      if (p.prob) p.prob[r] = (float)share_of(to_float(row[token]), best, heat, total);
    }
  }
  if (dist) {
    const double inv = (double)(1ull << kFix) / (double)total;
    const float ih = (float)inv, il = (float)(inv - (double)ih);
    for_tokens(row, lo, hi, [&](float x, int i) {
      float v = 0.f, yh, yl;
      s.w.orders(x, yh, yl);
      if (x >= w.floor && yh < 152.f && place_of(x, i) >= kept) {
        float a, b;
        int n;
        pow2_neg(sm.pow2, yh, yl, a, b, n);
        const float h = a * ih;
        v = h + (fmaf(a, ih, -h) + fmaf(a, il, b * ih));
        // (in two steps, of which only the second may leave the normal numbers)
        const int m = min(n, 100);
        v = v * __int_as_float((127 - m) << 23) * __int_as_float((127 - (n - m)) << 23);
      }
      dist[i] = v;
    });
  }
  cluster.sync();
}

// One warp per sequence: the first row whose draft does not stay.
__global__ void __launch_bounds__(256) accept_kernel(const SampleParams p) {
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
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.rows * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, int sms, cudaStream_t st) {
  // CTAs of a row: as many as fill the SMs once, with 2048 tokens each at least
  int ctas = 1;
  while (ctas < kMaxCluster && (long long)p.rows * ctas * 2 <= sms && p.vocab >= 4096 * ctas) ctas *= 2;
  cudaError_t e = p.rows == 0             ? cudaSuccess
                  : p.type == KVR_ACT_F32 ? launch<float>(p, ctas, st)
                  : p.type == KVR_ACT_BF16 ? launch<__nv_bfloat16>(p, ctas, st)
                                           : launch<__half>(p, ctas, st);
  if (e != cudaSuccess || !p.cu) return e;
  accept_kernel<<<(p.n_seq + 7) / 8, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace kvr
