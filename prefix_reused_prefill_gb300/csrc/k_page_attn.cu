// Attention over the 4-bit pages for sequences with few rows (kvr_page_attend):
// one-token steps and speculative verify.
//
//   o_r = sum_k p_rk v_k / sum_k p_rk,   p_rk = 2^(scale log2(e) q_r k_k - m_r)
// over the keys k that row r sees, with the running maximum m_r of one pass.
// With k_k = sK_kj (c - 8) per group j of 32 dims, the score is
//   sum_j sK_kj (sum_(d in j) q_d c_kd - 8 sum_(d in j) q_d).
// The tensor cores multiply the 4-bit codes themselves: a nibble in bits 0-3
// (4-7) of a 16-bit half IS the fp16 subnormal c 2^-24 (c 2^-20), one AND per
// two codes.  (Their sums align a subnormal as if it were 2^-14 in size, which
// costs a score at most 2^-13 of max|q| sK: measured, 2^-14 of the term.)  The
// scale multiplies the fp32 sum of its group.
// The values are summed over thousands of keys, where such a cut and the bias of
// 8 would add up: there a code becomes the fp16 number c - 8 (the nibble under
// the exponent of 1024 or 64, less 1032 or 72: exact), and
//   o_d = sum_k (p_k sV_kj) (c_kd - 8)
// with the scale on the weights: p and p sV are fp16 (2^-11 each, relative to
// the weight; the row's sum takes p unrounded), p held with a factor 4 so that
// p sV stays in range (p <= 1, sV <= 8188).  q is scaled per row by a power of
// two so that any bf16 q is an fp16 number.
//
// Keys are the M side of both products (m16n8k16, S^T = K Q^T and O^T = V^T P^T):
// the rows, at most 8 or 16 of a tile, fill the narrow N side.
//
// Bound by HBM: a page of one KV head is 9216 contiguous bytes (head dim 128),
// fetched by one bulk copy.  The work, all (sequence, row tile, KV head, page)
// units in this order, is cut into equal runs, one for each CTA and in it one
// for each warp, whatever the lengths are; every warp streams its run through a
// ring of its own.  A segment (the pages of one sequence, tile and head) that
// one warp covers alone is finished by it; otherwise the warps' parts are
// merged by the CTA, and the CTAs' parts by the last of them to arrive, in the
// order of the pages.
#include "kvr_pages.cuh"

namespace kvr {

namespace {

constexpr int kWarps = kPageAttnWarps;
constexpr int kThreads = 32 * kWarps;

template <int D, int NT>
struct Cfg {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kGroups = D / 32;
  static constexpr int kChunk = Chunk<D>::kBytes;
  static constexpr int kRows = 8 * NT;
  static constexpr int kRing = kStages * kChunk;
  static constexpr int kSlot = kPageAttnRows * D;   // floats of a partial result
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// d += a (16x16 fp16) * b (16x8 fp16)
__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  __half2 r = __hadd2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
// codes in bits 0-3 and 4-7 of both halves as the fp16 numbers c - 8
__device__ __forceinline__ uint32_t centred_lo(uint32_t w) {
  return hadd2((w & 0x000f000fu) | 0x64006400u, 0xe408e408u);   // 1024 + c - 1032
}
__device__ __forceinline__ uint32_t centred_hi(uint32_t w) {
  return hadd2((w & 0x00f000f0u) | 0x54005400u, 0xd480d480u);   // 64 + c - 72
}
template <int W>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t* w) {
  if (W == 4) {
    const uint4 v = dev::lds128(addr);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  }
}
// the scales of one key's groups
template <int W>
__device__ __forceinline__ void lds_scales(uint32_t addr, float* s) {
  if (W == 4) {
    uint32_t a, b;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr));
    const float2 x = dev::act2<true>(a), y = dev::act2<true>(b);
    s[0] = x.x; s[1] = x.y; s[2] = y.x; s[3] = y.y;
  } else {
    const float2 x = dev::act2<true>(dev::lds32(addr));
    s[0] = x.x; s[1] = x.y;
  }
}

// A segment and the place of a unit in it.
struct Place {
  int b, tile, kv, page;   // sequence, row tile, KV head, page of the sequence
  int pages;               // pages of the segment
  int row0, m, P;          // first row and rows of the sequence, its tokens before them
};

// a partial result: [rows of a tile][D] floats, and (m, l) per row
struct Slot {
  float* o;
  float2* ml;
};

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(kThreads, 1) page_attn_kernel(const PagesDev p, const PageAttend a) {
  using C = Cfg<D, NT>;
  using K = Chunk<D>;
  constexpr int kG = C::kGroups;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[kWarps][C::kStages];
  __shared__ int first_unit[kPageMaxSeqs + 1];   // units before each sequence
  __shared__ int scan[kWarps];
  // partial results of this CTA in the order of the pages: two per warp
  __shared__ int rec_seg[2 * kWarps];            // first unit of the segment, -1 for none
  __shared__ int rec_seg_n[2 * kWarps];          // its units
  __shared__ int last_flag;
  __shared__ int abort_flag;
  volatile int* abort_v = &abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;

  dev::pdl_trigger();
  if (tid < kWarps * C::kStages) dev::mbar_init(dev::smem_u32(&full_bar[0][0] + tid), 1);
  if (tid < 2 * kWarps) rec_seg[tid] = -1;
  if (tid < kWarps * C::kStages) dev::fence_mbar_init();
  dev::pdl_wait();
  if (tid == 0) abort_flag = dev::status_set(p.status) ? 1 : 0;

  // ---- units before every sequence
  const int n = p.info[0];
  const int rows_all = min(a.rows, p.info[1]);
  auto seq_rows = [&](int b) { return max(0, min(p.cu[b + 1], rows_all) - p.cu[b]); };
  int carry = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int b = base + tid;
    int u = 0;
    if (b < n) {
      const int m = seq_rows(b);
      if (m > 0 && p.G * m <= a.many)
        u = ((p.G * m + C::kRows - 1) / C::kRows) * p.Hkv * ((p.lens[b] + kPage - 1) / kPage);
    }
    int inc = u;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += scan[w];
      carry += scan[w];
    }
    if (b < n) first_unit[b] = before + inc - u;
  }
  if (tid == 0) first_unit[n] = carry;
  __syncthreads();
  const int units = carry;
  if (units == 0 || *abort_v) return;
  // every warp gets a unit before another CTA is taken
  const int ctas = min((int)gridDim.x, (units + kWarps - 1) / kWarps);
  const int cta = blockIdx.x;
  if (cta >= ctas) return;
  const int c0 = (int)((long long)units * cta / ctas), c1 = (int)((long long)units * (cta + 1) / ctas);
  const int w0 = c0 + (int)((long long)(c1 - c0) * warp / kWarps);
  const int w1 = c0 + (int)((long long)(c1 - c0) * (warp + 1) / kWarps);

  auto place_of = [&](int u) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_unit[mid] <= u) lo = mid;
      else hi = mid;
    }
    Place s;
    s.b = lo;
    s.m = seq_rows(lo);
    s.row0 = p.cu[lo];
    const int len = p.lens[lo];
    // the sequence's rows by the plan, some of which may lie past the buffers
    s.P = len - (p.cu[lo + 1] - s.row0);
    s.pages = (len + kPage - 1) / kPage;
    const int r = u - first_unit[lo];
    s.page = r % s.pages;
    s.kv = (r / s.pages) % p.Hkv;
    s.tile = r / s.pages / p.Hkv;
    return s;
  };
  // output row (token, query head) of row r of a tile, -1 past the last
  auto out_row = [&](const Place& s, int r) -> long long {
    const int rho = s.tile * C::kRows + r;
    if (rho >= p.G * s.m) return -1;
    return (long long)(s.row0 + rho / p.G) * p.Hq + s.kv * p.G + rho % p.G;
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
  // partial results: [gridDim.x][2 kWarps] of the warps, then [gridDim.x][2] of the CTAs
  auto warp_slot = [&](int i) {
    const long long at = (long long)cta * 2 * kWarps + i;
    return Slot{a.part + at * C::kSlot, a.ml + at * kPageAttnRows};
  };
  auto cta_slot = [&](int c, int i) {
    const long long at = (long long)gridDim.x * 2 * kWarps + (long long)c * 2 + i;
    return Slot{a.part + at * C::kSlot, a.ml + at * kPageAttnRows};
  };

  // ---- this warp's run
  bool ok = true;
  if (w0 < w1) {
    const uint32_t ring = dev::smem_u32(smem) + warp * C::kRing;
    const uint32_t bars = dev::smem_u32(&full_bar[warp][0]);
    const uint8_t* layer = p.pool + p.layer_off;
    // addresses of the next 32 units to fetch, one per lane
    long long src = 0;
    int queued = w0;   // first unit past the queue
    int issued = w0;
    auto issue = [&]() {
      if (issued == queued) {
        const int u = queued + lane;
        if (u < w1) {
          const Place s = place_of(u);
          src = ((long long)p.table[(long long)s.b * p.width + s.page] * p.Hkv + s.kv) * C::kChunk;
        }
        queued += 32;
      }
      const long long off = __shfl_sync(0xffffffffu, src, (issued - w0) & 31);
      if (lane == 0) {
        const int st = (issued - w0) % C::kStages;
        dev::mbar_arrive_expect_tx(bars + 8 * st, C::kChunk);
        bulk_load(ring + st * C::kChunk, layer + off, C::kChunk, bars + 8 * st);
      }
      ++issued;
    };
    while (issued < w1 && issued - w0 < C::kStages) issue();

    Place s = place_of(w0);
    uint32_t qb[NT][kG][4];       // dims 32 j + 8 t + 0..7 of row 8 n + g, the B side of the K codes
    float bias[NT][kG][2];        // -8 sum of q over the group, rows 8 n + 2 t, + 1 (units 2^-20)
    float f[NT][2];               // sums -> scores in log2 units
    int see[NT][2];               // last key these rows see
    float m_run[NT][2], l_run[NT][2];
    float o[NT][2 * kG][4];       // O^T tiles 2 j, 2 j + 1: rows g, g + 8 are dims 32 j + 4 g + 0, 1 and + 2, 3
    bool fresh = true;
    int part_no = 0;              // partial results of this warp so far

    for (int u = w0; u < w1 && ok; ++u) {
      if (fresh) {
        fresh = false;
#pragma unroll
        for (int nn = 0; nn < NT; ++nn) {
          // row 8 nn + g of the tile: this lane's dims of it
          const int rho = s.tile * C::kRows + 8 * nn + g;
          uint4 raw[kG];
          const bool live = rho < p.G * s.m;
#pragma unroll
          for (int j = 0; j < kG; ++j) {
            raw[j] = make_uint4(0, 0, 0, 0);
            if (live)
              raw[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                       (long long)(s.row0 + rho / p.G) * a.qs +
                                                       (s.kv * p.G + rho % p.G) * D + 32 * j + 8 * t);
          }
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
          // 2^e with |q| 2^e in [2^10, 2^11); e from the exponent field, kept
          // where both 2^e and its inverse are normal numbers.  The nibble in
          // bits 0-3 counts 2^-24, so its q carries another factor of 16.
          int e = 137 - (int)(__float_as_uint(top) >> 23);
          e = top > 0.f ? max(-100, min(100, e)) : 0;
          const float up = __uint_as_float((uint32_t)(127 + e) << 23);
          float neg[kG];
#pragma unroll
          for (int j = 0; j < kG; ++j) {
            const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 x = dev::act2<F16>(w[i]);
              const __half2 h = __floats2half2_rn(x.x * up, x.y * up);
              const float2 hf = __half22float2(h);
              sum += hf.x + hf.y;
              qb[nn][j][i] = i & 1 ? *reinterpret_cast<const uint32_t*>(&h)
                                   : dev::pack_act<true>(hf.x * 16.f, hf.y * 16.f);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            neg[j] = sum * (-8.f / 1048576.f);
          }
          const float back = __uint_as_float((uint32_t)(127 - e) << 23) * 1048576.f * a.scale_log2;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int from = (2 * t + c) * 4;
#pragma unroll
            for (int j = 0; j < kG; ++j) bias[nn][j][c] = __shfl_sync(0xffffffffu, neg[j], from);
            f[nn][c] = __shfl_sync(0xffffffffu, back, from);
            const int rc = s.tile * C::kRows + 8 * nn + 2 * t + c;
            see[nn][c] = rc < p.G * s.m ? s.P + rc / p.G : -1;
            m_run[nn][c] = -INFINITY;
            l_run[nn][c] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 2 * kG; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[nn][i][c] = 0.f;
        }
      }
      const int st = (u - w0) % C::kStages;
      ok = dev::mbar_wait(bars + 8 * st, ((u - w0) / C::kStages) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok && !*abort_v);
      if (!ok) break;
      const uint32_t page = ring + st * C::kChunk;
      const int key_base = s.page * kPage;
      // every row of the tile sees the whole page
      const bool whole = key_base + kPage <= s.P + 1;

      // ---- scores of 64 keys
      float sc[4][NT][4];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t w0k[kG], w1k[kG];
        float s0[kG], s1[kG];
        lds_words<kG>(page + K::k_word(16 * mt + g, t, 0), w0k);
        lds_words<kG>(page + K::k_word(16 * mt + 8 + g, t, 0), w1k);
        lds_scales<kG>(page + K::k_scale(16 * mt + g, 0), s0);
        lds_scales<kG>(page + K::k_scale(16 * mt + 8 + g, 0), s1);
#pragma unroll
        for (int nn = 0; nn < NT; ++nn)
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[mt][nn][c] = 0.f;
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          const uint32_t x0 = w0k[j], x1 = w1k[j], y0 = x0 >> 8, y1 = x1 >> 8;
          const uint32_t a0 = x0 & 0x000f000fu, a1 = x1 & 0x000f000fu, a2 = x0 & 0x00f000f0u,
                         a3 = x1 & 0x00f000f0u;
          const uint32_t b0 = y0 & 0x000f000fu, b1 = y1 & 0x000f000fu, b2 = y0 & 0x00f000f0u,
                         b3 = y1 & 0x00f000f0u;
#pragma unroll
          for (int nn = 0; nn < NT; ++nn) {
            float acc[4] = {bias[nn][j][0], bias[nn][j][1], bias[nn][j][0], bias[nn][j][1]};
            mma(acc, a0, a1, a2, a3, qb[nn][j][0], qb[nn][j][1]);
            mma(acc, b0, b1, b2, b3, qb[nn][j][2], qb[nn][j][3]);
            sc[mt][nn][0] = fmaf(acc[0], s0[j], sc[mt][nn][0]);
            sc[mt][nn][1] = fmaf(acc[1], s0[j], sc[mt][nn][1]);
            sc[mt][nn][2] = fmaf(acc[2], s1[j], sc[mt][nn][2]);
            sc[mt][nn][3] = fmaf(acc[3], s1[j], sc[mt][nn][3]);
          }
        }
      }
      // ---- running maximum and weights
      uint32_t pw[4][NT][2];
#pragma unroll
      for (int nn = 0; nn < NT; ++nn) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float x = sc[mt][nn][c] * f[nn][c & 1];
            if (!whole && key_base + 16 * mt + g + 8 * (c >> 1) > see[nn][c & 1]) x = -INFINITY;
            sc[mt][nn][c] = x;
            mx[c & 1] = fmaxf(mx[c & 1], x);
          }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], d));
        const bool moved = mx[0] > m_run[nn][0] || mx[1] > m_run[nn][1];
        if (__any_sync(0xffffffffu, moved)) {
          float corr[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float m_new = fmaxf(m_run[nn][c], mx[c]);
            corr[c] = m_run[nn][c] == -INFINITY ? 0.f : exp2f(m_run[nn][c] - m_new);
            m_run[nn][c] = m_new;
            l_run[nn][c] *= corr[c];
          }
#pragma unroll
          for (int i = 0; i < 2 * kG; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[nn][i][c] *= corr[c & 1];
        }
        // weights with a factor of 4 (in O and in l alike)
        float sub[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) sub[c] = m_run[nn][c] == -INFINITY ? 0.f : m_run[nn][c] - 2.f;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          float e[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            e[c] = ex2_approx(sc[mt][nn][c] - sub[c & 1]);
            l_run[nn][c & 1] += e[c];
          }
          pw[mt][nn][0] = transpose8x8(dev::pack_act<true>(e[0], e[1]));
          pw[mt][nn][1] = transpose8x8(dev::pack_act<true>(e[2], e[3]));
        }
      }
      // ---- weighted values
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
          const uint32_t e0 = centred_lo(x0), e1 = centred_hi(x0), e2 = centred_lo(x1), e3 = centred_hi(x1);
          const uint32_t f0 = centred_lo(y0), f1 = centred_hi(y0), f2 = centred_lo(y1), f3 = centred_hi(y1);
#pragma unroll
          for (int nn = 0; nn < NT; ++nn) {
            uint32_t b0 = hmul2(pw[mt][nn][0], s0[j]), b1 = hmul2(pw[mt][nn][1], s1[j]);
            if (!whole) {
              // a weight of zero takes nothing, whatever stands in a place
              // behind the row's last key (an unwritten scale, a NaN)
              const uint32_t p0 = pw[mt][nn][0], p1 = pw[mt][nn][1];
              b0 &= ((p0 & 0xffffu) ? 0xffffu : 0u) | ((p0 >> 16) ? 0xffff0000u : 0u);
              b1 &= ((p1 & 0xffffu) ? 0xffffu : 0u) | ((p1 >> 16) ? 0xffff0000u : 0u);
            }
            mma(o[nn][2 * j], e0, e1, e2, e3, b0, b1);
            mma(o[nn][2 * j + 1], f0, f1, f2, f3, b0, b1);
          }
        }
      }
      __syncwarp();
      if (issued < w1) issue();

      // ---- the end of the segment or of the run
      const bool seg_end = s.page + 1 == s.pages;
      if (seg_end || u + 1 == w1) {
        const int seg0 = u - s.page;
        const bool alone = seg_end && seg0 >= w0;
        const int rec = 2 * warp + part_no;
        const Slot out = warp_slot(rec);
#pragma unroll
        for (int nn = 0; nn < NT; ++nn) {
          float l[2], inv[2];
          long long row[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            l[c] = l_run[nn][c];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
            // (a NaN sum stays one)
            inv[c] = alone ? (l[c] == 0.f ? 0.f : 1.f / l[c]) : 1.f;
            row[c] = alone ? out_row(s, 8 * nn + 2 * t + c) : 0;
          }
#pragma unroll
          for (int j = 0; j < kG; ++j) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float x = o[nn][2 * j][c] * inv[c], y = o[nn][2 * j][2 + c] * inv[c];
              const float z = o[nn][2 * j + 1][c] * inv[c], w = o[nn][2 * j + 1][2 + c] * inv[c];
              if (alone) {
                if (row[c] >= 0) store4(row[c], 32 * j + 4 * g, x, y, z, w);
              } else {
                *reinterpret_cast<float4*>(out.o + (8 * nn + 2 * t + c) * D + 32 * j + 4 * g) =
                    make_float4(x, y, z, w);
              }
            }
          }
          if (!alone && g == 0) {
#pragma unroll
            for (int c = 0; c < 2; ++c) out.ml[8 * nn + 2 * t + c] = make_float2(m_run[nn][c], l[c]);
          }
        }
        if (!alone) {
          if (lane == 0) {
            rec_seg[rec] = seg0;
            rec_seg_n[rec] = s.pages;
          }
          ++part_no;
        }
        fresh = true;
        if (u + 1 < w1) s = place_of(u + 1);
      } else {
        ++s.page;
      }
    }
    if (!ok) {
      // a wait gave up: the copies in flight still land in this CTA's memory
      *abort_v = 1;
      const unsigned long long deadline = dev::globaltimer_ns() + kWaitLimitNs;
      for (int st = 0; st < C::kStages && st < issued - w0; ++st) {
        const int last = ((issued - 1 - w0 - st) / C::kStages) * C::kStages + st;
        dev::mbar_wait_until(bars + 8 * st, (uint32_t)(last / C::kStages) & 1, deadline);
      }
    }
  }
  __threadfence_block();
  __syncthreads();
  if (*abort_v) return;

  // ---- merge the warps' parts, then the CTAs': `count` parts given by
  // slot(i), element (row, 4 dims) after element
  auto merge = [&](int count, auto slot, auto done) {
    for (int e = tid; e < C::kRows * (D / 4); e += kThreads) {
      const int r = e / (D / 4), d = 4 * (e % (D / 4));
      float m = -INFINITY;
      for (int i = 0; i < count; ++i) m = fmaxf(m, __ldcg(&slot(i).ml[r]).x);
      float l = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < count; ++i) {
        const Slot s = slot(i);
        const float2 ml = __ldcg(s.ml + r);
        const float4 y = __ldcg(reinterpret_cast<const float4*>(s.o + r * D + d));
        // a part in which the row saw nothing (m = -inf, or -inf throughout
        // because its scores are NaN) counts its sum and its values as they are
        const float w = ml.x == -INFINITY ? 1.f : exp2f(ml.x - m);
        l = fmaf(w, ml.y, l);
        x.x = fmaf(w, y.x, x.x);
        x.y = fmaf(w, y.y, x.y);
        x.z = fmaf(w, y.z, x.z);
        x.w = fmaf(w, y.w, x.w);
      }
      done(r, d, x, m, l);
    }
  };
  auto finish = [&](const Place& s) {
    return [&, s](int r, int d, float4 x, float m, float l) {
      const long long row = out_row(s, r);
      if (row < 0) return;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      store4(row, d, x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    };
  };
  for (int i = 0; i < 2 * kWarps;) {
    const int seg0 = rec_seg[i];
    if (seg0 < 0) {
      ++i;
      continue;
    }
    // the records of one segment, in order; empty ones between them are skipped
    const int first = i, seg_n = rec_seg_n[i];
    int count = 0;
    uint32_t used = 0;
    for (; i < 2 * kWarps && (rec_seg[i] < 0 || rec_seg[i] == seg0); ++i)
      if (rec_seg[i] == seg0) {
        used |= 1u << (i - first);
        ++count;
      }
    const Place s = place_of(seg0);
    auto mine = [&](int k) { return warp_slot(first + (int)__fns(used, 0, k + 1)); };
    if (seg0 >= c0 && seg0 + seg_n <= c1) {
      merge(count, mine, finish(s));
      continue;
    }
    // the CTAs of the segment: the one that holds its first unit leaves its
    // part in its second slot, the others in their first
    auto owner = [&](int u) { return (int)(((long long)(u + 1) * ctas - 1) / units); };
    const int ca = owner(seg0), cb = owner(seg0 + seg_n - 1);
    const Slot out = cta_slot(cta, cta == ca ? 1 : 0);
    merge(count, mine, [&](int r, int d, float4 x, float m, float l) {
      *reinterpret_cast<float4*>(out.o + r * D + d) = x;
      if (d == 0) out.ml[r] = make_float2(m, l);
    });
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      last_flag = dev::atom_add_acq_rel(a.counters + ca, 1) == cb - ca;
      if (last_flag) a.counters[ca] = 0;
    }
    __syncthreads();
    if (last_flag) {
      __threadfence();
      merge(cb - ca + 1, [&](int k) { return cta_slot(ca + k, k == 0 ? 1 : 0); }, finish(s));
    }
    __syncthreads();
  }
}

template <int D, int NT, bool F16>
cudaError_t setup_one() {
  return cudaFuncSetAttribute(page_attn_kernel<D, NT, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kWarps * Cfg<D, NT>::kRing);
}
template <int D, int NT, bool F16>
cudaError_t launch_one(const PagesDev& p, const PageAttend& a, int ctas, cudaStream_t st) {
  return launch_k(page_attn_kernel<D, NT, F16>, dim3(ctas), kThreads, (size_t)kWarps * Cfg<D, NT>::kRing, st, p, a);
}

}  // namespace

cudaError_t page_attn_setup() {
  cudaError_t e = setup_one<128, 1, false>();
  if (e == cudaSuccess) e = setup_one<128, 2, false>();
  if (e == cudaSuccess) e = setup_one<64, 1, false>();
  if (e == cudaSuccess) e = setup_one<64, 2, false>();
  if (e == cudaSuccess) e = setup_one<128, 1, true>();
  if (e == cudaSuccess) e = setup_one<128, 2, true>();
  if (e == cudaSuccess) e = setup_one<64, 1, true>();
  if (e == cudaSuccess) e = setup_one<64, 2, true>();
  return e;
}

cudaError_t launch_page_attn(const PagesDev& p, const PageAttend& a, int nt, int ctas, cudaStream_t st) {
  if (p.d == 128) {
    if (p.f16) return nt == 1 ? launch_one<128, 1, true>(p, a, ctas, st) : launch_one<128, 2, true>(p, a, ctas, st);
    return nt == 1 ? launch_one<128, 1, false>(p, a, ctas, st) : launch_one<128, 2, false>(p, a, ctas, st);
  }
  if (p.f16) return nt == 1 ? launch_one<64, 1, true>(p, a, ctas, st) : launch_one<64, 2, true>(p, a, ctas, st);
  return nt == 1 ? launch_one<64, 1, false>(p, a, ctas, st) : launch_one<64, 2, false>(p, a, ctas, st);
}

}  // namespace kvr
