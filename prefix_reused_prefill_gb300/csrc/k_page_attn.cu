// Attention over the 4-bit pages for sequences with few rows (kvr_page_attend):
// one-token steps and speculative verify.
//
//   o_r = sum_k p_rk v_k / sum_k p_rk,   p_rk = 2^(scale log2(e) q_r k_k - m_r)
// over the keys k that row r sees, with the running maximum m_r of one pass.
// With k_k = sK_kj (c - 8) per group j of 32 dims, the score is the sum over j of
// sK_kj (sum_(d in j) q_d (c_kd - 8)), and with v_k = sV_kj (c - 8)
//   o_d = sum_k (p_k sV_kj) (c_kd - 8).
// The tensor cores multiply the codes, as fp16 numbers c - 8: the nibble under the
// exponent of 1024 or 64 (one AND-OR for two codes), less 1032 or 72, exactly.
// (The nibble alone is an fp16 subnormal and needs no subtraction, but sums of
// such products are cut at 2^-14 of the code unit, and with the bias of 8 that
// adds up over thousands of keys.)  The K scale multiplies the fp32 sum of its
// group, the V scale the codes: (c - 8) sV and p are fp16 (2^-11 each, relative to
// themselves; the row's sum takes p unrounded).  (c - 8) sV loses nothing where it is
// small, as sV is a multiple of 2^-24 itself, and p has a factor of 2^15, so that what fp16
// drops is below 2^-38 of the largest weight in a run: attention stays linear in V.
// (p sV instead has a quarter of the products with sV and took 71.8 instead of 74 us in
// the first example below, but lost weights below 2^-27 / sV: the tail under a sink.)
// q is scaled per row by a power of two that brings its largest element to 2^10, and is fp16.
//
// Keys are the M side of both products (m16n8k16, S^T = K Q^T and O^T = V^T P^T):
// the rows, at most 8 of a tile, fill the narrow N side.
//
// Bound by HBM: a page of one KV head is 9216 contiguous bytes (head dim 128),
// fetched as two bulk copies, K and V.  The work, all (sequence, row tile, KV
// head, page) units in this order, is cut into equal runs, one for each CTA and
// in it one for each warp, whatever the lengths are; every warp streams its run
// through a ring of its own.  A segment (the pages of one sequence, tile and
// head) that one warp covers alone is finished by it; otherwise the warps'
// parts are merged by the CTA, and the CTAs' parts by the last of them to
// arrive, in the order of the pages.  Where there are few segments, each of a
// page or two per warp, a CTA takes a whole one instead: the second page costs
// less than a merge across CTAs.
//
// 64 sequences of one token over up to 8191 (32 heads in groups of 4, d = 128): 74 us,
// 3.9 TB/s of 289 MB, 58 % of a plain copy's rate (a bare streaming loop over the
// same pages: 6.3 TB/s).  Two over 131070 (28 heads in groups of 7): 48 us, 3.2 TB/s.
// Of both about 3 us go before the first page and 5 to 8 us to the last pages, the
// parts and their merge; between them an SM takes about 415 cycles a page, 300 at
// the copy's rate.  One sequence over 726: 10.0 us.  Four of 8 rows over 15360
// (groups of 7): 55 us, where seven tiles of 8 rows each decode the pages anew.
#include <cfloat>
#include <climits>

#include "kvr_pages.cuh"

namespace kvr {

namespace {

using dev::ex2_approx;
using dev::hadd2;
using dev::held;
using dev::hmul2;
using dev::number2;

// 16 warps: one alone waits for its loads and products most of the time.  (Tiles of
// 16 rows, with the registers of 8 warps, take 830 cycles a page instead of 430 and
// had half the warps for start and merge: 14 rows over 15360 tokens 51 us, 19 so.)
template <int D>
struct Cfg {
  static constexpr int kWarps = 16;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kGroups = D / 32;
  static constexpr int kHalf = Chunk<D>::kHalf;
  static constexpr int kStages = 48 / kWarps * (128 / D);   // halves of pages
  static constexpr int kRows = 8;
  static constexpr int kRing = kStages * kHalf;
  static constexpr int kSlot = kRows * D;                   // floats of a partial result
  static_assert(kSlot * 4 + kRows * 8 <= kRing, "a partial result fits the ring");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// d += a (16x16 fp16) * b (16x8 fp16).  (Not volatile, and the loads below are
// ordinary ones: the compiler interleaves the products of several keys and dims
// with the loads and decoding of the next.)
__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = a * b
__device__ __forceinline__ void mma_first(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// the halves of a pair that the first n of two stand for
__device__ __forceinline__ uint32_t first_of_pair(int n) { return n > 1 ? 0xffffffffu : n == 1 ? 0xffffu : 0u; }
// codes in bits 0-3 (4-7) of both halves as the fp16 numbers c - 8; k1024 and k64
// hold those numbers in both halves
template <uint32_t kMask>
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "n"(kMask), "r"(bits));
  return r;
}
__device__ __forceinline__ uint32_t centred_lo(uint32_t w, uint32_t k1024) {
  return hadd2(and_or<0x000f000fu>(w, k1024), 0xe408e408u);   // 1024 + c - 1032
}
__device__ __forceinline__ uint32_t centred_hi(uint32_t w, uint32_t k64) {
  return hadd2(and_or<0x00f000f0u>(w, k64), 0xd480d480u);     // 64 + c - 72
}
template <int W>
__device__ __forceinline__ void sts_words(uint8_t* at, const uint32_t* w) {
  if (W == 4) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[W - 2], w[W - 1]);
  else *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
}
template <int W>
__device__ __forceinline__ void lds_words(const uint8_t* at, uint32_t* w) {
  if (W == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    w[0] = v.x; w[1] = v.y;
  }
}
// the scales of one key's groups
template <int W>
__device__ __forceinline__ void lds_scales(const uint8_t* at, float* s) {
  if (W == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    const float2 x = dev::act2<true>(v.x), y = dev::act2<true>(v.y);
    s[0] = x.x; s[1] = x.y; s[2] = y.x; s[3] = y.y;
  } else {
    const float2 x = dev::act2<true>(*reinterpret_cast<const uint32_t*>(at));
    s[0] = x.x; s[1] = x.y;
  }
}

// A segment and the place of a unit in it.
struct Place {
  int b, tile, kv, page;   // sequence, row tile, KV head, page of the sequence
  int pages;               // pages of the segment
  int row0, m, P;          // first row and rows of the sequence, its tokens before them
};

// the segment of a partial result: its units, and the rows it belongs to
struct Rec {
  int pages, tile, kv, row0, m;
};

template <int N>
struct Vec {
  float v[N];
  float2 xy;
};
// N neighbouring floats, not from L1
template <int N>
__device__ __forceinline__ Vec<N> load_past_l1(const void* p) {
  Vec<N> r;
  if (N == 4) {
    asm volatile("ld.relaxed.gpu.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(r.v[0]), "=f"(r.v[1]), "=f"(r.v[N - 2]), "=f"(r.v[N - 1])
                 : "l"(p)
                 : "memory");
  } else {
    asm volatile("ld.relaxed.gpu.v2.f32 {%0, %1}, [%2];" : "=f"(r.v[0]), "=f"(r.v[1]) : "l"(p) : "memory");
  }
  r.xy = make_float2(r.v[0], r.v[1]);
  return r;
}

// a partial result: [rows of a tile][D] floats, and per row the exponent that its
// weights are taken under and their sum
struct Slot {
  float* o;
  float2* ml;
};

// Merge the parts of the segments that CTAs of the tensor-memory kernel share:
// a warp takes two rows, a lane D / 32 dims of each, and the loads of four parts of
// both are in flight together (four rows: 41 instead of 33 us where 84 rows over
// 15360 tokens have parts of 60 CTAs).  The whole grid shares the rows of all segments.
template <int D, bool F16>
__device__ void merge_tc(const PagesDev& p, const PageAttend& a, int warp_id, int warps) {
  constexpr int kPer = D / 32, kRows = 2, kGroups = kPageTcRows / kRows;
  const int lane = threadIdx.x & 31, r0 = kRows * (warp_id % kGroups);
  // the segments that start in CTAs first, first + step, ..; a lane looks at each
  const int first = warp_id / kGroups, step = warps / kGroups;
  const int mine = first + step * lane;
  uint32_t todo = __ballot_sync(0xffffffffu, mine < (int)gridDim.x && a.shared[mine].parts > 0);
  for (; todo; todo &= todo - 1) {
    const int ca = first + step * (__ffs(todo) - 1);
    const PageShared s = a.shared[ca];
    const int rows = min(kPageTcRows, s.R - kPageTcRows * s.tile);
    if (r0 >= rows) continue;
    float m[kRows], l[kRows], x[kRows][kPer];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      m[q] = -INFINITY;
      l[q] = 0.f;
#pragma unroll
      for (int d = 0; d < kPer; ++d) x[q][d] = 0.f;
    }
#pragma unroll 4
    for (int k = 0; k < s.parts; ++k) {
      const long long at = ((long long)(ca + k) * 2 + (k == 0 ? 1 : 0)) * kPageTcRows + r0;
      float2 ml[kRows];
      float y[kRows][kPer];
#pragma unroll
      for (int q = 0; q < kRows; ++q) {   // (a slot has whole tiles of rows)
        ml[q] = __ldcg(a.tc_ml + at + q);
        const float* src = a.tc_part + (at + q) * D + kPer * lane;
        if (kPer == 4) {
          const float4 z = __ldcg(reinterpret_cast<const float4*>(src));
          y[q][0] = z.x; y[q][1] = z.y; y[q][kPer - 2] = z.z; y[q][kPer - 1] = z.w;
        } else {
          const float2 z = __ldcg(reinterpret_cast<const float2*>(src));
          y[q][0] = z.x; y[q][1] = z.y;
        }
      }
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
        // (a part in which the row saw nothing counts as it is: zeros, or NaN)
        const float m_new = fmaxf(m[q], ml[q].x);
        const float old = m[q] == m_new ? 1.f : ex2_approx(m[q] - m_new);
        const float w = ml[q].x == -INFINITY ? 1.f : ex2_approx(ml[q].x - m_new);
        m[q] = m_new;
        l[q] = fmaf(l[q], old, w * ml[q].y);
#pragma unroll
        for (int d = 0; d < kPer; ++d) x[q][d] = fmaf(x[q][d], old, w * y[q][d]);
      }
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      if (r0 + q >= rows) break;
      const float inv = l[q] == 0.f ? 0.f : 1.f / l[q];
      const int rho = kPageTcRows * s.tile + r0 + q;
      const int tok = (int)((uint32_t)rho / (uint32_t)p.G);
      uint16_t* dst = static_cast<uint16_t*>(a.out) +
                      ((long long)(s.row0 + tok) * p.Hq + s.kv * p.G + rho - tok * p.G) * D + kPer * lane;
      uint32_t v[kPer / 2];
#pragma unroll
      for (int d = 0; d < kPer; d += 2)
        v[d / 2] = F16 || !a.out_f16 ? dev::pack_act<F16>(x[q][d] * inv, x[q][d + 1] * inv)
                                     : dev::pack_act2(x[q][d] * inv, x[q][d + 1] * inv, true);
      if (kPer == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(v[0], v[kPer / 2 - 1]);
      else *reinterpret_cast<uint32_t*>(dst) = v[0];
    }
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
page_attn_kernel(const PagesDev p, const PageAttend a) {
  using C = Cfg<D>;
  using K = Chunk<D>;
  constexpr int kG = C::kGroups, kWarps = C::kWarps, kThreads = C::kThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[kWarps][C::kStages];
  __shared__ int first_unit[kPageMaxSeqs + 1];   // units before each sequence
  __shared__ int scan_u[kWarps], scan_s[kWarps], scan_p[kWarps];
  // partial results of this CTA in the order of the pages: two per warp, one in
  // the work area (a segment that ended inside the run) and one in its ring
  __shared__ int rec_seg[2 * kWarps];            // first unit of the segment, -1 for none
  __shared__ Rec rec_of[2 * kWarps];
  __shared__ int rec_list[2 * kWarps], seg_at[2 * kWarps + 1], seg_count;
  __shared__ int own[2];                         // this CTA's run
  __shared__ int last_flag[2];
  __shared__ int abort_flag;
  volatile int* abort_v = &abort_flag;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int cta = blockIdx.x;

  dev::pdl_trigger();
  if (tid < kWarps * C::kStages) {
    dev::mbar_init(dev::smem_u32(&full_bar[0][0] + tid), 1);
    dev::fence_mbar_init();
  }
  if (tid < 2 * kWarps) rec_seg[tid] = -1;
  dev::pdl_wait();
  if (tid == 0) abort_flag = dev::status_set(p.status) ? 1 : 0;

  // ---- units before every sequence.  (The first sequences' values are asked for
  // along with the number of sequences: any entry of the tables can be read.)
  int row0 = 0, row1 = 0, len = 0;
  auto fetch = [&](int b) {
    if (b < p.max_seqs) {
      row0 = p.cu[b];
      row1 = p.cu[b + 1];
      len = p.lens[b];
    }
  };
  fetch(tid);
  const int n = p.info[0];
  const int rows_all = min(a.rows, p.info[1]);
  int units = 0, segs = 0, most_pages = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int b = base + tid;
    int u = 0, sg = 0, pages = 0;
    if (base) fetch(b);
    const int m = min(row1, rows_all) - row0;
    // (the launch, captured under another plan, knew of no sequence so long)
    if (cta == 0 && b < n && p.G * m > a.many && !a.shared && *p.refused == 0) *p.refused = KVR_ERR_UNSUPPORTED;
    if (b < n && m > 0 && p.G * m <= a.many) {
      pages = (len + kPage - 1) / kPage;
      sg = ((p.G * m + C::kRows - 1) / C::kRows) * p.Hkv;
      u = sg * pages;
    }
    int iu = u, is = sg;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int ou = __shfl_up_sync(0xffffffffu, iu, d), os = __shfl_up_sync(0xffffffffu, is, d);
      if (lane >= d) {
        iu += ou;
        is += os;
      }
    }
    const int mp = __reduce_max_sync(0xffffffffu, pages);
    __syncthreads();
    if (lane == 31) {
      scan_u[warp] = iu;
      scan_s[warp] = is;
      scan_p[warp] = mp;
    }
    __syncthreads();
    int before_u = units, before_s = segs;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        before_u += scan_u[w];
        before_s += scan_s[w];
      }
      units += scan_u[w];
      segs += scan_s[w];
      most_pages = max(most_pages, scan_p[w]);
    }
    if (b < n) first_unit[b] = before_u + iu - u;
    // the segment of this CTA, should each CTA take one
    const int k = cta - (before_s + is - sg);
    if (k >= 0 && k < sg) {
      own[0] = before_u + iu - u + k * pages;
      own[1] = own[0] + pages;
    }
  }
  if (tid == 0) first_unit[n] = units;
  __syncthreads();
  if (*abort_v) return;
  if (a.shared) merge_tc<D, F16>(p, a, cta * kWarps + warp, (int)gridDim.x * kWarps);
  if (units == 0) return;
  const bool whole_segs = segs <= (int)gridDim.x && most_pages <= 2 * kWarps;
  // else every warp gets a unit before another CTA is taken
  const int ctas = whole_segs ? segs : min((int)gridDim.x, (units + kWarps - 1) / kWarps);
  if (cta >= ctas) return;
  // runs of `each` units, the first `odd` CTAs' one longer
  const int each = (int)((uint32_t)units / (uint32_t)ctas), odd = units - each * ctas;
  const int c0 = whole_segs ? own[0] : each * cta + min(cta, odd);
  const int c1 = whole_segs ? own[1] : c0 + each + (cta < odd ? 1 : 0);
  const int w0 = c0 + (c1 - c0) * warp / kWarps;   // (a run has less than 2^27 units)
  const int w1 = c0 + (c1 - c0) * (warp + 1) / kWarps;

  auto place_of = [&](int u) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_unit[mid] <= u) lo = mid;
      else hi = mid;
    }
    Place s;
    const int row0 = p.cu[lo], row1 = p.cu[lo + 1], len = p.lens[lo];
    s.b = lo;
    s.row0 = row0;
    s.m = min(row1, rows_all) - row0;
    // (the sequence's rows by the plan, some of which may lie past the buffers)
    s.P = len - (row1 - row0);
    s.pages = (len + kPage - 1) / kPage;
    const uint32_t r = u - first_unit[lo], seg = r / (uint32_t)s.pages;
    s.page = r - seg * s.pages;
    s.tile = dev::div_by(seg, p.mul_hkv);
    s.kv = seg - s.tile * p.Hkv;
    return s;
  };
  // the next segment
  auto advance = [&](Place& s) {
    s.page = 0;
    if (++s.kv < p.Hkv) return;
    s.kv = 0;
    if (C::kRows * ++s.tile < p.G * s.m) return;
    int u = first_unit[s.b + 1];
    do ++s.b;
    while (first_unit[s.b + 1] == u);
    s = place_of(u);
  };
  // row r of a tile: its token in the sequence and head in the group
  auto token_of = [&](int rho) { return dev::div_by(rho, p.mul_g); };
  // output row (token, query head) of row r of a tile, -1 past the last
  auto out_row = [&](int tile, int kv, int row0, int m, int r) -> long long {
    const int rho = tile * C::kRows + r;
    if (rho >= p.G * m) return -1;
    const int tok = token_of(rho);
    return (long long)(row0 + tok) * p.Hq + kv * p.G + rho - tok * p.G;
  };
  auto store4 = [&](long long row, int d, float x, float y, float z, float w) {
    uint2 v;
    if (F16 || !a.out_f16) {
      v = make_uint2(dev::pack_act<F16>(x, y), dev::pack_act<F16>(z, w));
    } else {
      v = make_uint2(dev::pack_act2(x, y, true), dev::pack_act2(z, w, true));
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + d) = v;
  };
  // partial results: in the work area [gridDim.x][kWarps] of the warps, then
  // [gridDim.x][2] of the CTAs
  auto global_slot = [&](long long at) { return Slot{a.part + at * C::kSlot, a.ml + at * C::kRows}; };
  auto warp_slot = [&](int i) {
    if (i & 1) {
      float* o = reinterpret_cast<float*>(smem + (i >> 1) * C::kRing);
      return Slot{o, reinterpret_cast<float2*>(o + C::kSlot)};
    }
    return global_slot((long long)cta * kWarps + (i >> 1));
  };
  auto cta_slot = [&](int c, int i) { return global_slot((long long)gridDim.x * kWarps + (long long)c * 2 + i); };

  // ---- this warp's run
  bool ok = true;
  if (w0 < w1) {
    const uint32_t ring = dev::smem_u32(smem) + warp * C::kRing;
    const uint32_t bars = dev::smem_u32(&full_bar[warp][0]);
    const uint8_t* layer = p.pool + p.layer_off;
    // chunks (page * KV heads + head) of the next 32 units to fetch, one per lane
    int src = 0;
    const int halves = 2 * (w1 - w0);
    int issued = 0;                       // halves requested
    uint32_t stage_in = 0;                // the stage of the next one, and its offset in the ring
    auto issue = [&]() {
      if ((issued & 63) == 0) {
        const int u = w0 + (issued >> 1) + lane;
        if (u < w1) {
          const Place s = place_of(u);
          src = p.table[(long long)s.b * p.width + s.page] * p.Hkv + s.kv;
        }
      }
      const uint8_t* from =
          layer + (long long)__shfl_sync(0xffffffffu, src, (issued >> 1) & 31) * K::kBytes + (issued & 1) * C::kHalf;
      if (lane == 0) {
        dev::mbar_arrive_expect_tx(bars + 8 * stage_in, C::kHalf);
        bulk_load(ring + stage_in * C::kHalf, from, C::kHalf, bars + 8 * stage_in);
      }
      ++issued;
      stage_in = stage_in + 1 == C::kStages ? 0 : stage_in + 1;
    };
    while (issued < halves && issued < C::kStages) issue();
    // the next half to use: its stage and the parity of that stage's phase
    uint32_t stage = 0, parity = 0;
    auto arrived = [&]() {
      if (__all_sync(0xffffffffu, dev::mbar_try_wait(bars + 8 * stage, parity))) return true;
      const bool got = dev::mbar_wait(bars + 8 * stage, parity, p.status) && !*abort_v;
      return (bool)__all_sync(0xffffffffu, got);
    };
    auto used = [&]() {
      __syncwarp();
      if (++stage == C::kStages) {
        stage = 0;
        parity ^= 1;
      }
      if (issued < halves) issue();
    };

    Place s = place_of(w0);
    uint32_t qb[kG][4];       // dims 32 j + 8 t + 0..7 of row 8 n + g, the B side of the K codes
    float f[2];               // sums -> scores in log2 units
    int see[2];               // last key these rows see
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2];
    // The exponent that a row's weights are taken under: 15 below the maximum, which fp16 has
    // room for (in O and in l alike).  Both are rounded up, so no weight passes 2^15, and the
    // largest, which often is most of the sum, is 2^15 without a rounding.
    auto ref_of = [](float m) { return __fadd_ru(m, -15.f); };
    float o[2 * kG][4];       // O^T tiles 2 j, 2 j + 1: rows g, g + 8 are dims 32 j + 4 g + 0, 1 and + 2, 3
    bool fresh = true;
    const uint32_t k1024 = held(0x64006400u), k64 = held(0x54005400u);

    // row g of the tile: this lane's dims of it
    auto load_q = [&](const Place& at, uint4* raw) {
      const int rho = at.tile * C::kRows + g;
      const int tok = token_of(rho);
      const uint16_t* src_q = static_cast<const uint16_t*>(a.q) + (long long)(at.row0 + tok) * a.qs +
                              (at.kv * p.G + rho - tok * p.G) * D + 8 * t;
#pragma unroll
      for (int j = 0; j < kG; ++j) {
        raw[j] = make_uint4(0, 0, 0, 0);
        if (rho < p.G * at.m) raw[j] = *reinterpret_cast<const uint4*>(src_q + 32 * j);
      }
    };
    // one page
    auto page_step = [&]() {
      const int key_base = s.page * kPage;
      // every row of the tile sees the whole page?
      const bool whole = key_base + kPage <= s.P + 1;
      if (!arrived()) return false;
      const uint8_t* page = smem + warp * C::kRing + stage * C::kHalf;
      // ---- scores of 64 keys
      float sc[4][4];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t w0k[kG], w1k[kG];
        float s0[kG], s1[kG];
        lds_words<kG>(page + K::k_word(16 * mt + g, t, 0), w0k);
        lds_words<kG>(page + K::k_word(16 * mt + 8 + g, t, 0), w1k);
        lds_scales<kG>(page + K::k_scale(16 * mt + g, 0), s0);
        lds_scales<kG>(page + K::k_scale(16 * mt + 8 + g, 0), s1);
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[mt][c] = 0.f;
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          const uint32_t x0 = w0k[j], x1 = w1k[j], y0 = x0 >> 8, y1 = x1 >> 8;
          const uint32_t a0 = centred_lo(x0, k1024), a1 = centred_lo(x1, k1024), a2 = centred_hi(x0, k64),
                         a3 = centred_hi(x1, k64);
          const uint32_t b0 = centred_lo(y0, k1024), b1 = centred_lo(y1, k1024), b2 = centred_hi(y0, k64),
                         b3 = centred_hi(y1, k64);
          float acc[4];
          mma_first(acc, a0, a1, a2, a3, qb[j][0], qb[j][1]);
          mma(acc, b0, b1, b2, b3, qb[j][2], qb[j][3]);
          sc[mt][0] = fmaf(acc[0], s0[j], sc[mt][0]);
          sc[mt][1] = fmaf(acc[1], s0[j], sc[mt][1]);
          sc[mt][2] = fmaf(acc[2], s1[j], sc[mt][2]);
          sc[mt][3] = fmaf(acc[3], s1[j], sc[mt][3]);
        }
      }
      used();
      if (!whole) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (key_base + 16 * mt + g + 8 * (c >> 1) > see[c & 1]) sc[mt][c] = -INFINITY;
      }
      // ---- running maximum and weights
      uint32_t pw[4][2];
      // (the factors f are positive: the maximum is taken before them)
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c & 1] = fmaxf(mx[c & 1], sc[mt][c]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], d));
        mx[c] = __fmul_ru(mx[c], f[c]);
      }
      const bool moved = mx[0] > m_run[0] || mx[1] > m_run[1];
      if (__any_sync(0xffffffffu, moved)) {
        float corr[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float m_new = fmaxf(m_run[c], mx[c]);
          if (m_new < -kScoreMax) m_new = -INFINITY;
          corr[c] = m_run[c] == -INFINITY ? 0.f : ex2_approx(ref_of(m_run[c]) - ref_of(m_new));
          m_run[c] = m_new;
          l_run[c] = m_new >= kScoreMax ? NAN : l_run[c] * corr[c];
        }
#pragma unroll
        for (int i = 0; i < 2 * kG; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[i][c] *= corr[c & 1];
      }
      float sub[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) sub[c] = m_run[c] == -INFINITY ? 0.f : ref_of(m_run[c]);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        float e[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          e[c] = ex2_approx(fmaf(sc[mt][c], f[c & 1], -sub[c & 1]));
          l_run[c & 1] += e[c];
        }
        pw[mt][0] = transpose8x8(dev::pack_act<true>(e[0], e[1]));
        pw[mt][1] = transpose8x8(dev::pack_act<true>(e[2], e[3]));
      }
      // ---- weighted values
      if (!arrived()) return false;
      if (!whole) {
        // Places behind the last token hold anything: no value.  A NaN among the scales of a
        // key, of which 0 times would reach every row, becomes the sum of the rows that see it.
        // (A lane looks at two keys' scales.  Little code: it is fetched anew nearly every time.)
        uint8_t* at = smem + warp * C::kRing + stage * C::kHalf + (K::kVs - C::kHalf) + lane * kG * 4;
        const int key = key_base + 16 * (lane >> 3) + 8 * (lane & 1) + (lane & 6);
        const uint32_t there = first_of_pair(s.P + s.m - key);
        uint32_t sv[kG], bad = 0;
        lds_words<kG>(at, sv);
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          bad |= (sv[j] & there) + 0x03ff03ffu;   // (bit 15 of a NaN's half)
          sv[j] = number2(sv[j] & there);
        }
        sts_words<kG>(at, sv);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the stage's next copy
        __syncwarp();
        const int first = __reduce_min_sync(0xffffffffu, bad & 0x8000u ? key : (int)bad < 0 ? key + 1 : INT_MAX);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (first <= see[c]) l_run[c] = NAN;
      }
      page = smem + warp * C::kRing + stage * C::kHalf - C::kHalf;   // (the V half's offsets count from the page)
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t v0[kG], v1[kG], s0[kG], s1[kG];
        lds_words<kG>(page + K::kV + ((2 * mt * 8 + g) * 4 + t) * kG * 4, v0);
        lds_words<kG>(page + K::kV + (((2 * mt + 1) * 8 + g) * 4 + t) * kG * 4, v1);
        lds_words<kG>(page + K::kVs + ((mt * 4 + t) * 2 + 0) * kG * 4, s0);
        lds_words<kG>(page + K::kVs + ((mt * 4 + t) * 2 + 1) * kG * 4, s1);
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          const uint32_t x0 = v0[j], x1 = v1[j], y0 = x0 >> 8, y1 = x1 >> 8;
          const uint32_t e0 = hmul2(centred_lo(x0, k1024), s0[j]), e1 = hmul2(centred_hi(x0, k64), s0[j]),
                         e2 = hmul2(centred_lo(x1, k1024), s1[j]), e3 = hmul2(centred_hi(x1, k64), s1[j]);
          const uint32_t f0 = hmul2(centred_lo(y0, k1024), s0[j]), f1 = hmul2(centred_hi(y0, k64), s0[j]),
                         f2 = hmul2(centred_lo(y1, k1024), s1[j]), f3 = hmul2(centred_hi(y1, k64), s1[j]);
          mma(o[2 * j], e0, e1, e2, e3, pw[mt][0], pw[mt][1]);
          mma(o[2 * j + 1], f0, f1, f2, f3, pw[mt][0], pw[mt][1]);
        }
      }
      used();
      return true;
    };

    for (int u = w0; u < w1 && ok; ++u) {
      if (fresh) {
        fresh = false;
        uint4 raw[kG];
        load_q(s, raw);
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = dev::act2<F16>(w[i]);
            top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
          }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e with max|q| 2^e in [2^10, 2^11), e from the exponent field, for every finite q
        // (-117 is that of the largest; 126 leaves 2^-e a normal number).
        // What is 2^-25 of the row's largest or more is exact, the rest is rounded by 2^-35 of it.
        int e = 137 - (int)(__float_as_uint(top) >> 23);
        e = top > 0.f ? max(-117, min(126, e)) : 0;
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = dev::act2<F16>(w[i]);
            qb[j][i] = dev::pack_act<true>(x.x * up, x.y * up);
          }
        }
        // (a number above 0, as masked scores of -inf are multiplied by it)
        const float back = fmaxf(__uint_as_float((uint32_t)(127 - e) << 23) * a.scale_log2, FLT_MIN);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int from = (2 * t + c) * 4;
          f[c] = __shfl_sync(0xffffffffu, back, from);
          const int rc = s.tile * C::kRows + 2 * t + c;
          see[c] = rc < p.G * s.m ? s.P + token_of(rc) : -1;
          m_run[c] = -INFINITY;
          l_run[c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2 * kG; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
      }
      ok = page_step();
      if (!ok) break;

      // ---- the end of the segment or of the run
      const bool seg_end = s.page + 1 == s.pages;
      if (seg_end || u + 1 == w1) {
        const int seg0 = u - s.page;
        const bool alone = seg_end && seg0 >= w0;
        const int rec = 2 * warp + (u + 1 == w1 ? 1 : 0);
        const Slot out = warp_slot(rec);
        float l[2], inv[2];
        long long row[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          l[c] = l_run[c];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
          // (a NaN sum stays one)
          inv[c] = alone ? (l[c] == 0.f ? 0.f : 1.f / l[c]) : 1.f;
          row[c] = alone ? out_row(s.tile, s.kv, s.row0, s.m, 2 * t + c) : 0;
        }
#pragma unroll
        for (int j = 0; j < kG; ++j) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float x = o[2 * j][c] * inv[c], y = o[2 * j][2 + c] * inv[c];
            const float z = o[2 * j + 1][c] * inv[c], w = o[2 * j + 1][2 + c] * inv[c];
            if (alone) {
              if (row[c] >= 0) store4(row[c], 32 * j + 4 * g, x, y, z, w);
            } else {
              *reinterpret_cast<float4*>(out.o + (2 * t + c) * D + 32 * j + 4 * g) =
                  make_float4(x, y, z, w);
            }
          }
        }
        if (!alone && g == 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c) out.ml[2 * t + c] = make_float2(ref_of(m_run[c]), l[c]);
        }
        if (!alone) {
          if (lane == 0) {
            rec_seg[rec] = seg0;
            rec_of[rec] = {s.pages, s.tile, s.kv, s.row0, s.m};
          }
        }
        fresh = true;
        if (u + 1 < w1) advance(s);
      } else {
        ++s.page;
      }
    }
    if (!ok) {
      // a wait gave up: the copies in flight still land in this CTA's memory
      *abort_v = 1;
      const unsigned long long deadline = dev::globaltimer_ns() + kWaitLimitNs;
      for (int st = 0; st < (int)C::kStages && st < issued; ++st) {
        const int last = (issued - 1 - st) / C::kStages;
        dev::mbar_wait_until(bars + 8 * st, (uint32_t)last & 1, deadline);
      }
    }
  }
  __syncthreads();
  if (*abort_v) return;

  // ---- merge the warps' parts, then the CTAs'
  auto owner = [&](int u) {
    const int longer = (each + 1) * odd;
    return u < longer ? u / (each + 1) : odd + (u - longer) / each;
  };
  // the filled records in order, and the first record of each segment
  static_assert(2 * kWarps <= 32, "one record per lane");
  if (warp == 0) {
    const bool has = lane < 2 * kWarps && rec_seg[lane] >= 0;
    uint32_t mask = __ballot_sync(0xffffffffu, has);
    const uint32_t below = (1u << lane) - 1;
    if (has) rec_list[__popc(mask & below)] = lane;
    const int records = __popc(mask);
    __syncwarp();
    const bool starts =
        lane < records && (lane == 0 || rec_seg[rec_list[lane]] != rec_seg[rec_list[lane - 1]]);
    mask = __ballot_sync(0xffffffffu, starts);
    if (starts) seg_at[__popc(mask & below)] = lane;
    if (lane == 0) {
      seg_count = __popc(mask);
      seg_at[__popc(mask)] = records;
    }
  }
  __syncthreads();
  int jobs = seg_count;
  if (jobs == 0) return;
  // First time round: the CTA's own parts of each segment, to the output or, where other
  // CTAs share it (the first and the last segment at most), to the work area.
  // Second time: what the last CTA to arrive finds there.  A warp takes a row, a lane
  // D / 32 dims of it.  (Reads go past L1: other CTAs wrote some of them.)
#pragma unroll 1
  for (int round = 0;; ++round) {
#pragma unroll 1
    for (int x = warp; x < jobs * C::kRows; x += kWarps) {
      const int k = x / C::kRows, r = x % C::kRows;
      if (round && !last_flag[k]) continue;
      const int first = seg_at[round && k ? seg_count - 1 : k], at = rec_list[first], seg0 = rec_seg[at];
      const Rec s = rec_of[at];
      const bool local = seg0 >= c0 && seg0 + s.pages <= c1;
      const int ca = round ? owner(seg0) : 0;
      const int count = round ? owner(seg0 + s.pages - 1) - ca + 1 : seg_at[k + 1] - first;
      constexpr int kPer = D / 32;
      float m = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
      for (int d = 0; d < kPer; ++d) o[d] = 0.f;
#pragma unroll 8
      for (int i = 0; i < count; ++i) {
        // (the CTA that holds a segment's first unit leaves its part in its
        // second slot, the others in their first)
        const Slot sl = round ? cta_slot(ca + i, i == 0 ? 1 : 0) : warp_slot(rec_list[first + i]);
        const float2 ml = load_past_l1<2>(sl.ml + r).xy;
        const Vec<kPer> y = load_past_l1<kPer>(sl.o + r * D + kPer * lane);
        // a part in which the row saw nothing (m = -inf, or -inf throughout
        // because its scores are NaN) counts its sum and its values as they are
        const float m_new = fmaxf(m, ml.x);
        const float old = m == m_new ? 1.f : ex2_approx(m - m_new);
        const float w = ml.x == -INFINITY ? 1.f : ex2_approx(ml.x - m_new);
        m = m_new;
        l = fmaf(l, old, w * ml.y);
#pragma unroll
        for (int d = 0; d < kPer; ++d) o[d] = fmaf(o[d], old, w * y.v[d]);
      }
      if (round || local) {
        const long long row = out_row(s.tile, s.kv, s.row0, s.m, r);
        if (row < 0) continue;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* dst = static_cast<uint16_t*>(a.out) + row * D + kPer * lane;
#pragma unroll
        for (int d = 0; d < kPer; d += 2)
          reinterpret_cast<uint32_t*>(dst)[d / 2] = F16 || !a.out_f16
                                                        ? dev::pack_act<F16>(o[d] * inv, o[d + 1] * inv)
                                                        : dev::pack_act2(o[d] * inv, o[d + 1] * inv, true);
      } else {
        const Slot out = cta_slot(cta, seg0 >= c0 ? 1 : 0);
#pragma unroll
        for (int d = 0; d < kPer; ++d) out.o[r * D + kPer * lane + d] = o[d];
        if (lane == 0) out.ml[r] = make_float2(m, l);
      }
    }
    if (round) return;
    // the first segment may have begun in an earlier CTA, the last may go on in
    // the next (one that does both counts as the first)
    const int s_first = rec_seg[rec_list[0]], s_last = rec_seg[rec_list[seg_at[seg_count - 1]]];
    const bool with_before = s_first < c0;
    const bool with_after = s_last >= c0 && s_last + rec_of[rec_list[seg_at[seg_count - 1]]].pages > c1;
    if (!with_before && !with_after) return;
    __syncthreads();   // (the add below releases what the CTA wrote)
    if (tid < 2) {
      last_flag[tid] = 0;
      if (tid ? with_after : with_before) {
        const int seg0 = tid ? s_last : s_first;
        const int ca = owner(seg0), cb = owner(seg0 + rec_of[rec_list[tid ? seg_at[seg_count - 1] : 0]].pages - 1);
        if (dev::atom_add_acq_rel(a.counters + ca, 1) == cb - ca) {
          a.counters[ca] = 0;
          last_flag[tid] = 1;
        }
      }
    }
    __syncthreads();
    if (!last_flag[0] && !last_flag[1]) return;
    jobs = 2;
  }
}

template <int D, bool F16>
cudaError_t setup_one() {
  using C = Cfg<D>;
  return cudaFuncSetAttribute(page_attn_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              C::kWarps * C::kRing);
}
template <int D, bool F16>
cudaError_t launch_one(const PagesDev& p, const PageAttend& a, int ctas, cudaStream_t st) {
  using C = Cfg<D>;
  return launch_k(page_attn_kernel<D, F16>, dim3(ctas), C::kThreads, (size_t)C::kWarps * C::kRing, st, p, a);
}

}  // namespace

cudaError_t page_attn_setup() {
  cudaError_t e = setup_one<128, false>();
  if (e == cudaSuccess) e = setup_one<64, false>();
  if (e == cudaSuccess) e = setup_one<128, true>();
  if (e == cudaSuccess) e = setup_one<64, true>();
  return e;
}

cudaError_t launch_page_attn(const PagesDev& p, const PageAttend& a, int ctas, cudaStream_t st) {
  if (p.d == 128) return p.f16 ? launch_one<128, true>(p, a, ctas, st) : launch_one<128, false>(p, a, ctas, st);
  return p.f16 ? launch_one<64, true>(p, a, ctas, st) : launch_one<64, false>(p, a, ctas, st);
}

}  // namespace kvr
