// Attention over the 4-bit pages for sequences with many rows (kvr_page_attend):
// suffix prefill and wide speculative verify, on the 5th-generation tensor cores.
//
// S = Q K^T and O += P V in blocks of 128 keys, softmax in one pass with a lazy
// running maximum (a row's O is rescaled only when its maximum grows by more
// than 2^8).  K and V become fp16 tiles in shared memory: c - 8 exactly (as in
// k_page_attn.cu), times the scale: a product of at most 14 bits.  For bf16
// activations it is rounded once (2^-11, an eighth of what the output's own type
// drops).  For fp16 that rounding would be as large as the output's, and the
// scores' twice as large, so K and V are two fp16 terms each, the second the exact rest
// of the first, and every product runs once for each: 5.6e-4 -> 2.6e-4 of the
// outputs in the mean square at scores of deviation 2 (2.1e-4 is the output's rounding), for
// 31.4 instead of 30.3 us in a mixed batch of 64-wide heads and 897 instead of 667 us
// in the long prompts below (twice the products, one stage of K and V, and 88 bytes a
// thread of spilled registers; the other forms spill 8 to 28).  q is scaled per row by a
// power of two that brings its largest element to 2^10 (what is 2^-25 of that or more is
// exact), and is fp16; P is fp16 with a factor of 2^7 (2^-11, and nothing above 2^-31 of
// the largest is lost).  Sums, maxima and O are fp32.  (The tensor core cuts its sums, so that
// with weights and values all alike an output is low by 0.2 % after a CTA's run of 0.44
// million keys, two terms each, and by 0.34 % after 1.8 million.)
//
// Writing a 4-bit block as fp16 costs about as many instructions as the softmax
// of one 128-row tile over it, so a CTA runs two row tiles over each block: one
// dequantisation feeds four products.  Tensor memory holds S (P over it) and O
// of both tiles, 512 columns; while the softmax of one tile runs, the tensor
// core works for the other.  Warp roles (20 warps, 96 registers a thread):
//   0-7, 8-15  softmax of tile 0 / 1, two threads per row, one for each 64 keys of
//              the block: S from tensor memory 8 keys at a time, weights under the
//              row's present reference, one vote of the two warps that share
//              rows whether a score passed it (then the reference moves and the
//              block is formed again), P back over the thread's own half of S.
//              Q into shared memory at the start of a segment.  The first warp
//              of a tile also issues the tile's products: its softmax, P V and
//              the next scores follow one another anyway.
//   16-19      a quarter of each block's keys, global -> registers (one block
//              ahead) -> the fp16 tiles: K [128 keys][d] and V as [d][128 keys]
//              (both K-major with the 128-byte swizzle), two stages each (one
//              where two terms of 128-wide heads fill the shared memory)
// The work, all (sequence, pair of row tiles, KV head, key block) units in this
// order, is cut into equal runs, one per CTA, whatever the lengths are; the parts
// of a segment (one sequence, pair and head) that several CTAs hold go to the
// work area, and the launch that follows (k_page_attn.cu) merges them with the
// whole card: one CTA took longer for that than for its run.
//
// A NaN scale: of K, it makes the key's score NaN.  Of V, it would reach rows
// that do not see the key (0 * NaN), so the key's score becomes NaN instead and
// the value 0: rows that see it read NaN.
// Every wait is bounded; a CTA whose wait gave up frees its tensor memory.
//
// Two prompts of up to 2047 rows over up to 14001 tokens (32 heads in groups of 4,
// d = 128, bf16, 766 GFLOP): 667 us, 1.15 PFLOP/s, 60 % of what a library product
// reaches.  A block of 128 keys takes a CTA about 4000 cycles, 2080 of them
// products.  Each tile's chain is what lasts so long: 2000 of softmax (1400 for the weights,
// the other tile and the writing warps on the same schedulers), 940 until P V is
// done (520 of products, the rest the commit's way to the waiting warp), which the next
// scores must wait for as they go over P, and 750 for them.  (Scores of the
// upper 64 keys issued before that wait, P all in the lower columns: 784 us, a
// product of 64 keys lasts as long as one of 128.  64-key blocks with two S:
// slower too.)
// 254 rows over 1668 tokens: 35.5 us, of which the run is about 11, the rest the start
// (6k cycles to the first product), Q, the parts' way to memory and the merge.
#include <cfloat>
#include <type_traits>

#include "kvr_pages.cuh"

namespace kvr {

namespace {

using dev::ex2_approx;
using dev::hadd2;
using dev::held;
using dev::hmul2;
using dev::number2;

constexpr int kTile = 128;
constexpr int kPairRows = kPageTcRows;
constexpr int kKeys = 128;
constexpr int kDecodeWarp = 16;
constexpr int kThreads = 32 * (kDecodeWarp + 4);
constexpr float kLazyMax = 8.0f;
// Weights carry a factor of 2^7 (in O and in l alike), so that the largest, 2^8 over the
// reference, is 2^15 and what fp16 drops is below 2^-31 of it.  Every rounding of a reference
// goes the way that no weight is larger.
constexpr float kHead = 7.0f;

template <int D, bool F16>
struct Tc {
  static constexpr int kTerms = F16 ? 2 : 1;     // fp16 terms of a K or V element
  static constexpr int kGroups = D / 32;
  static constexpr int kQTile = kTile * D * 2;   // d / 64 atoms of [128 rows][64 dims]
  static constexpr int kQAtom = kTile * 128;
  static constexpr int kKTerm = kKeys * D * 2;   // d / 64 atoms of [128 keys][64 dims]
  static constexpr int kKTile = kTerms * kKTerm;
  static constexpr int kKAtom = kKeys * 128;
  static constexpr int kVTerm = D * kKeys * 2;   // 2 atoms of [d dims][64 keys]
  static constexpr int kVTile = kTerms * kVTerm;
  static constexpr int kVAtom = D * 128;
  static constexpr int kStages = F16 && D == 128 ? 1 : 2;
  static constexpr int kSmem = 2 * kQTile + kStages * (kKTile + kVTile) + 1024;
};
// tensor memory columns
__device__ __forceinline__ uint32_t s_col(int t) { return (uint32_t)(128 * t); }
__device__ __forceinline__ uint32_t o_col(int t) { return (uint32_t)(256 + 128 * t); }

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// The low word of the descriptor of a tile with the 128-byte swizzle; the high word
// is the same for all (8 rows of 128 bytes apart, version 1, that swizzle).
constexpr uint32_t kDescHigh = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t sw128_desc(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }
__device__ __forceinline__ uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// A warp that issues products runs as one (every lane the same control flow, the elected
// lane's instructions predicated), so that the operands stay in uniform
// registers: from a branch of one lane each product cost about 117 cycles to
// issue instead of the 64 that it takes.
__device__ __forceinline__ uint32_t elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ void mma_ss(uint32_t elected, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "mov.b64 x, {%1, %6};\n\t"
      "mov.b64 y, {%2, %6};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(elected), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t elected, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "mov.b64 y, {%2, %6};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(elected), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t elected, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar),
      "r"(elected)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// barrier of n threads; whether p holds for any of them
__device__ __forceinline__ bool any_of(int id, int n, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)p)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void named_sync(int id, int n) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// a b - c, rounded once
__device__ __forceinline__ uint32_t hfms2(uint32_t a, uint32_t b, uint32_t c) {
  __half2 r = __hfma2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b),
                      __hneg2(*reinterpret_cast<__half2*>(&c)));
  return *reinterpret_cast<uint32_t*>(&r);
}
// the four code pairs of a word as fp16 numbers c - 8, times s: rounded, and what
// the rounding dropped (a number of at most 4 bits; 2^-24 is the least)
template <int kTerms>
struct Pairs {
  uint32_t v[kTerms][4];
};
template <int kTerms>
__device__ __forceinline__ Pairs<kTerms> decode(uint32_t w, uint32_t s, uint32_t k1024, uint32_t k64) {
  const uint32_t y = w >> 8;
  uint32_t a, b, c, d;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(a) : "r"(w), "r"(k1024));
  asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(b) : "r"(w), "r"(k64));
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(c) : "r"(y), "r"(k1024));
  asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(d) : "r"(y), "r"(k64));
  const uint32_t x[4] = {hadd2(a, 0xe408e408u), hadd2(b, 0xd480d480u), hadd2(c, 0xe408e408u), hadd2(d, 0xd480d480u)};
  Pairs<kTerms> p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p.v[0][i] = hmul2(x[i], s);
    if (kTerms == 2) p.v[kTerms - 1][i] = hfms2(x[i], s, p.v[0][i]);
  }
  return p;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// a word per group from global memory
template <int W>
__device__ __forceinline__ void ldg_words(const uint8_t* p, uint32_t* w) {
  if (W == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  }
}

// A segment: one sequence, pair of row tiles and KV head.
struct Seg {
  int b, tile, kv;
  int row0, m, P, len, R;   // the sequence's first row, rows, tokens before them, tokens; G * rows
  int nb;                   // key blocks that the pair's rows see
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
page_attn_tc_kernel(const PagesDev p, const PageAttendTc a) {
  using C = Tc<D, F16>;
  using K = Chunk<D>;
  constexpr int kG = C::kGroups, kTerms = C::kTerms, kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full[2], s_full[2], p_full[2], pv_done[2], drained[2];
  __shared__ __align__(8) uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  __shared__ long long first_unit[kPageMaxSeqs + 1];   // units before each sequence
  __shared__ int start[4];                             // this CTA's first unit: sequence, tile, head, block
  __shared__ uint32_t tmem_slot;
  __shared__ float exchange[2][2][kTile];              // [tile][half of the block][row]
  __shared__ int abort_flag;
  volatile int* abort_v = &abort_flag;
  // (the shuffle tells the compiler that a warp's number is one for its lanes)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int cta = blockIdx.x;
  const uint32_t base = (dev::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_base = base, k_base = q_base + 2 * C::kQTile, v_base = k_base + kStages * C::kKTile;

  dev::pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      dev::mbar_init(dev::smem_u32(&q_full[i]), 8);
      dev::mbar_init(dev::smem_u32(&s_full[i]), 1);
      dev::mbar_init(dev::smem_u32(&p_full[i]), 8);
      dev::mbar_init(dev::smem_u32(&pv_done[i]), 1);
      dev::mbar_init(dev::smem_u32(&drained[i]), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      dev::mbar_init(dev::smem_u32(&k_full[i]), 4);
      dev::mbar_init(dev::smem_u32(&k_empty[i]), 2);   // (one for each tile)
      dev::mbar_init(dev::smem_u32(&v_full[i]), 4);
      dev::mbar_init(dev::smem_u32(&v_empty[i]), 2);
    }
    dev::fence_mbar_init();
  }
  dev::pdl_wait();
  if (tid == 0) *abort_v = dev::status_set(p.status) ? 1 : 0;

  // ---- units before every sequence: a warp per sequence sums its pairs' blocks
  // (the first sequences' values are asked for along with their number)
  const int ahead = min(warp, p.max_seqs - 1);
  const int ahead0 = p.cu[ahead], ahead1 = p.cu[ahead + 1], ahead_len = p.lens[ahead];
  const int n = p.info[0];
  const int rows_all = min(a.rows, p.info[1]);
  auto set_seq = [&](Seg& s, int b, int row0, int row1, int len) {
    s.b = b;
    s.row0 = row0;
    s.m = max(0, min(row1, rows_all) - row0);
    s.len = len;
    s.P = len - (row1 - row0);
    s.R = p.G * s.m;
  };
  auto load_seq = [&](int b, Seg& s) {
    set_seq(s, b, p.cu[b], p.cu[b + 1], p.lens[b]);
    return s.R > a.many;
  };
  auto blocks_of = [&](const Seg& s, int tile) {
    const int last = (int)((uint32_t)(min(s.R, kPairRows * (tile + 1)) - 1) / (uint32_t)p.G);
    return (s.P + last + kKeys) / kKeys;
  };
  for (int b = warp; b < n; b += kThreads / 32) {
    Seg s;
    long long u = 0;
    if (b == warp) set_seq(s, b, ahead0, ahead1, ahead_len);
    else load_seq(b, s);
    if (s.R > a.many)
      for (int r = lane; r < (s.R + kPairRows - 1) / kPairRows; r += 32) u += blocks_of(s, r);
#pragma unroll
    for (int d = 16; d; d >>= 1) u += __shfl_xor_sync(0xffffffffu, u, d);
    if (lane == 0) first_unit[b] = u * p.Hkv;
  }
  __syncthreads();
  if (warp == 0) {
    // exclusive sums in place
    long long carry = 0;
    for (int b0 = 0; b0 < n; b0 += 32) {
      const int b = b0 + lane;
      const long long u = b < n ? first_unit[b] : 0;
      long long inc = u;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      if (b < n) first_unit[b] = carry + inc - u;
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) first_unit[n] = carry;
  }
  __syncthreads();
  const long long units = first_unit[n];
  auto describe = [&](const PageShared& x) {
    if (tid == 0) a.shared[cta] = x;
  };
  if (units == 0 || *abort_v) {
    describe(PageShared{});
    return;
  }
  const int ctas = units >= (long long)gridDim.x * a.min_units ? (int)gridDim.x
                                                               : ((int)units + a.min_units - 1) / a.min_units;
  if (cta >= ctas) {
    describe(PageShared{});
    return;
  }
  // runs of `each` units, the first `odd` of them one longer
  const long long each = units < (1ll << 31) ? (uint32_t)units / (uint32_t)ctas : units / ctas;
  const int odd = (int)(units - each * ctas);
  const long long c0 = each * cta + min(cta, odd), c1 = c0 + each + (cta < odd ? 1 : 0);
  auto owner = [&](long long u) {
    const long long longer = (each + 1) * odd;
    return (int)(u < longer ? u / (each + 1) : odd + (u - longer) / each);
  };
  // the segment that holds unit u, found by one warp
  auto locate = [&](long long u) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_unit[mid] <= u) lo = mid;
      else hi = mid;
    }
    Seg s;
    load_seq(lo, s);
    long long rem = u - first_unit[lo];
    for (int r0 = 0;; r0 += 32) {
      const int r = r0 + lane;
      const long long w = r < (s.R + kPairRows - 1) / kPairRows ? (long long)blocks_of(s, r) * p.Hkv : 0;
      long long inc = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, inc > rem);
      if (past) {
        const int at = __ffs(past) - 1;
        s.tile = r0 + at;
        rem -= __shfl_sync(0xffffffffu, inc - w, at);
        break;
      }
      rem -= __shfl_sync(0xffffffffu, inc, 31);
    }
    s.nb = blocks_of(s, s.tile);
    s.kv = (int)((uint32_t)rem / (uint32_t)s.nb);   // (rem < blocks * heads of a pair)
    start[0] = s.b;
    start[1] = s.tile;
    start[2] = s.kv;
    start[3] = (int)rem - s.kv * s.nb;
  };
  if (warp == 0) locate(c0);
  if (warp == kDecodeWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(dev::smem_u32(&tmem_slot)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  Seg first_seg;
  load_seq(start[0], first_seg);
  first_seg.tile = start[1];
  first_seg.kv = start[2];
  first_seg.nb = blocks_of(first_seg, first_seg.tile);
  const int first_block = start[3];
  auto advance = [&](Seg& s) {
    if (++s.kv < p.Hkv) return;
    s.kv = 0;
    if (kPairRows * (s.tile + 1) < s.R) {
      ++s.tile;
    } else {
      s.tile = 0;
      int b = s.b + 1;
      while (!load_seq(b, s)) ++b;   // (there is one: the run is not over)
    }
    s.nb = blocks_of(s, s.tile);
  };
  // body(segment, first block, last block + 1) for each segment of the run,
  // until it returns false
  auto for_segments = [&](auto body) {
    Seg s = first_seg;
    int j = first_block;
    for (long long u = c0; u < c1;) {
      const int je = (int)min((long long)s.nb, j + (c1 - u));
      if (!body(s, j, je)) return false;
      u += je - j;
      j = 0;
      if (u < c1) advance(s);
    }
    return true;
  };
  auto wait = [&](uint64_t& bar, uint32_t parity) {
    return dev::mbar_wait(dev::smem_u32(&bar), parity & 1, p.status) && !*abort_v;
  };
  // (the first look apart: with every look asking for the abort flag too, two
  // prompts of 2047 rows over up to 14001 tokens, 766 GFLOP, took 835 us
  // instead of 773)
  auto all_wait = [&](uint64_t& bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, dev::mbar_try_wait(dev::smem_u32(&bar), parity & 1))) return true;
    return (bool)__all_sync(0xffffffffu, wait(bar, parity));
  };
  // both of two waits, the first look at them together
  auto all_wait2 = [&](uint64_t& bar, uint32_t parity, uint64_t& bar2, uint32_t parity2) {
    const bool one = dev::mbar_try_wait(dev::smem_u32(&bar), parity & 1);
    const bool two = dev::mbar_try_wait(dev::smem_u32(&bar2), parity2 & 1);
    if (__all_sync(0xffffffffu, one && two)) return true;
    return all_wait(bar, parity) && all_wait(bar2, parity2);
  };
  bool ok = true;
  if (warp >= kDecodeWarp) {
    // ---------------------------------------------------------------- tiles
    // K: a lane has dims 32 j + 8 t .. + 7 of a key; lanes 0-3 and 4-7 of a
    // store hold keys 4 apart, whose chunks the swizzle puts side by side.
    // V: a lane has dims 32 j + 4 g .. + 3 of 8 keys (kb).
    const int w = warp - kDecodeWarp;
    const int t = lane & 3, key_in = (lane >> 3) | (lane & 4);
    const int g = lane >> 2, kb = 4 * w + (lane & 3), kbp = kb & 7;
    const uint32_t k1024 = held(0x64006400u), k64 = held(0x54005400u);
    uint32_t it = 0;
    ok = for_segments([&](const Seg& s, int j0, int j1) {
      const int32_t* table = p.table + (long long)s.b * p.width;
      const int pages = (s.len + kPage - 1) / kPage;
      const uint8_t* layer = p.pool + p.layer_off + (long long)s.kv * K::kBytes;
      // this warp's half page of block j (-1: past the sequence or the run)
      auto page_of = [&](int j) {
        const int pg = 2 * j + (w >> 1);
        return j < j1 && pg < pages ? table[pg] : -1;
      };
      uint32_t kc[4][kG], ks[4][kG / 2], kvs[4];   // K codes, scales, a scale of the key's value
      uint32_t vc[4][kG], vs[4][kG];               // V codes, scales
      auto fetch_k = [&](int pg) {
        const uint8_t* chunk = layer + (long long)pg * p.Hkv * K::kBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = 32 * (w & 1) + 8 * i + key_in;
          if (pg >= 0) {
            ldg_words<kG>(chunk + K::k_word(key, t, 0), kc[i]);
            const uint32_t* sp = reinterpret_cast<const uint32_t*>(chunk + K::k_scale(key, 0));
#pragma unroll
            for (int j = 0; j < kG / 2; ++j) ks[i][j] = sp[j];
            kvs[i] = *reinterpret_cast<const uint16_t*>(chunk + K::v_scale(key, t & (kG - 1)));
          } else {
#pragma unroll
            for (int j = 0; j < kG; ++j) kc[i][j] = 0;
#pragma unroll
            for (int j = 0; j < kG / 2; ++j) ks[i][j] = 0;
            kvs[i] = 0;
          }
        }
      };
      auto fetch_v = [&](int pg) {
        const uint8_t* chunk = layer + (long long)pg * p.Hkv * K::kBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (pg >= 0) {
            ldg_words<kG>(chunk + K::kV + ((kbp * 8 + g) * 4 + i) * kG * 4, vc[i]);
            ldg_words<kG>(chunk + K::kVs + (((kbp >> 1) * 4 + i) * 2 + (kbp & 1)) * kG * 4, vs[i]);
          } else {
#pragma unroll
            for (int j = 0; j < kG; ++j) vc[i][j] = vs[i][j] = 0;
          }
        }
      };
      int next_page = page_of(j0);
      fetch_k(next_page);
      fetch_v(next_page);
      next_page = page_of(j0 + 1);
      for (int j = j0; j < j1; ++j, ++it) {
        if (it >= kStages && !all_wait(k_empty[it % kStages], it / kStages - 1)) return false;
        const uint32_t k_tile = k_base + (it % kStages) * C::kKTile;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = 32 * w + 8 * i + key_in;
          // a NaN among the scales of the key's value
          const uint32_t nan = __ballot_sync(0xffffffffu, (kvs[i] & 0x7fffu) > 0x7c00u);
          const bool bad = (nan >> (lane & 28)) & 15u;
#pragma unroll
          for (int jj = 0; jj < kG; ++jj) {
            uint32_t s2 = __byte_perm(ks[i][jj / 2], 0, jj & 1 ? 0x3232 : 0x1010);
            if (bad) s2 = 0x7fff7fffu;
            const Pairs<kTerms> x = decode<kTerms>(kc[i][jj], s2, k1024, k64);
#pragma unroll
            for (int m = 0; m < kTerms; ++m)
              sts128(k_tile + m * C::kKTerm + (jj >> 1) * C::kKAtom + dev::swz128(key, 4 * (jj & 1) + t), x.v[m][0],
                     x.v[m][1], x.v[m][2], x.v[m][3]);
          }
        }
        fence_smem();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_u32(&k_full[it % kStages]));
        if (j + 1 < j1) fetch_k(next_page);
        if (it >= kStages && !all_wait(v_empty[it % kStages], it / kStages - 1)) return false;
        const uint32_t v_tile = v_base + (it % kStages) * C::kVTile + (kb >> 3) * C::kVAtom;
        // keys past the sequence weigh nothing and must not be NaN
        const int left = s.len - (kKeys * j + 8 * kb);
        if (left < 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t keep = (2 * i < left ? 0xffffu : 0u) | (2 * i + 1 < left ? 0xffff0000u : 0u);
#pragma unroll
            for (int jj = 0; jj < kG; ++jj) vs[i][jj] &= keep;
          }
        }
#pragma unroll
        for (int jj = 0; jj < kG; ++jj) {
          Pairs<kTerms> x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = decode<kTerms>(vc[i][jj], number2(vs[i][jj]), k1024, k64);
#pragma unroll
          for (int m = 0; m < kTerms; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sts128(v_tile + m * C::kVTerm + dev::swz128(32 * jj + 4 * g + e, kbp), x[0].v[m][e], x[1].v[m][e],
                     x[2].v[m][e], x[3].v[m][e]);
        }
        fence_smem();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_u32(&v_full[it % kStages]));
        if (j + 1 < j1) {
          fetch_v(next_page);
          next_page = page_of(j + 2);
        }
      }
      return true;
    });
  } else {
    // ---------------------------------------------------------------- softmax
    const int t = warp >> 3, h = (warp >> 2) & 1;   // row tile, half of the block's keys (and of O's dims)
    const int r = 32 * (warp & 3) + lane;           // row of the tile
    const int pair = 1 + 4 * t + (warp & 3);        // barrier of the two warps with the same rows
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_addr = lanes + s_col(t) + 64 * h, o_addr = lanes + o_col(t) + D / 2 * h;
    const uint32_t q_tile = q_base + t * C::kQTile;
    uint32_t blocks = 0;                            // blocks of this tile so far
    uint32_t it = 0, segs = 0;                      // all blocks of the run; segments of this tile
    const bool issuer = (warp & 7) == 0;
    const uint32_t el = elect();
    const uint32_t id_qk = idesc_f16(kTile, kKeys), id_pv = idesc_f16(kTile, D);
    // S = Q K^T of block i of the run; each tile frees the K stage
    auto scores = [&](uint32_t i) {
      const uint32_t qd = sw128_desc(q_tile), kd = sw128_desc(k_base + (i % kStages) * C::kKTile);
#pragma unroll
      for (int m = 0; m < kTerms; ++m)
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(el, tmem + s_col(t), qd + (kk >> 2) * (C::kQAtom >> 4) + 2 * (kk & 3),
                 kd + m * (C::kKTerm >> 4) + (kk >> 2) * (C::kKAtom >> 4) + 2 * (kk & 3), id_qk,
                 m > 0 || kk > 0 ? 1u : 0u);
      commit(el, dev::smem_u32(&s_full[t]));
      commit(el, dev::smem_u32(&k_empty[i % kStages]));
    };
    // ok stays false once a wait gave up: the warp then skips its work but
    // still meets its partner at every barrier
    for_segments([&](const Seg& s, int j0, int j1) {
      const int rho0 = kPairRows * s.tile + kTile * t;
      if (rho0 >= s.R) {
        // one tile only: the other's issuer passes every stage on unread.  (It
        // must not run ahead: a phase is told by its parity, so a wait is good
        // for the stage's present or next use only.)
        for (int j = j0; issuer && j < j1 && ok; ++j, ++it) {
          ok = all_wait(k_full[it % kStages], it / kStages);
          if (lane == 0 && ok) dev::mbar_arrive(dev::smem_u32(&k_empty[it % kStages]));
          ok = ok && all_wait(v_full[it % kStages], it / kStages);
          if (lane == 0 && ok) dev::mbar_arrive(dev::smem_u32(&v_empty[it % kStages]));
        }
        return true;
      }
      // every warp of the tile is done with the last segment: with the exchange
      // and with its part of the Q tile, which O went through
      named_sync(9 + t, 256);
      const int rho = rho0 + r;
      const bool live = rho < s.R;
      const int tok = live ? (int)((uint32_t)rho / (uint32_t)p.G) : 0;
      float f;
      {
        // q, scaled by a power of two with max|q| 2^e in [2^10, 2^11), as fp16: as
        // it is into the tile first, then in place.  (Short loops: code that runs
        // once is paid for by its fetch from memory, 16 bytes an instruction.)
        constexpr int kHalfChunks = D / 16;        // 16-byte chunks of half a row
        const uint32_t atom = q_tile + (D == 128 ? h * C::kQAtom : 0);
        const int first = D == 128 ? 0 : 4 * h;    // chunk within the 64 dims of an atom
        // a warp's 32 half rows, whole lines at a time
#pragma unroll 1
        for (int i = 0; i < kHalfChunks; ++i) {
          const int rr = 32 * (warp & 3) + 32 / kHalfChunks * i + lane / kHalfChunks, c = lane % kHalfChunks;
          const int rho2 = min(rho0 + rr, s.R - 1);
          const int tok2 = (int)((uint32_t)rho2 / (uint32_t)p.G);
          const uint16_t* src = static_cast<const uint16_t*>(a.q) + (long long)(s.row0 + tok2) * a.qs +
                                (s.kv * p.G + rho2 - tok2 * p.G) * D + D / 2 * h + 8 * c;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(atom + rr * 128 +
                                                                             (((first + c) ^ (rr & 7)) << 4)),
                       "l"(src), "r"(rho0 + rr < s.R ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        const uint32_t row = atom + r * 128;
        float top = 0.f;
#pragma unroll 2
        for (int c = 0; c < kHalfChunks; ++c) {
          const uint4 u = dev::lds128(row + (((first + c) ^ (r & 7)) << 4));
          const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 y = dev::act2<F16>(x[i]);
            top = max3(top, fabsf(y.x), fabsf(y.y));
          }
        }
        exchange[t][h][r] = top;
        named_sync(pair, 64);
        top = fmaxf(top, exchange[t][h ^ 1][r]);
        int e = 137 - (int)(__float_as_uint(top) >> 23);
        e = top > 0.f ? max(-117, min(126, e)) : 0;
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        // (a number above 0, as masked scores of -inf are multiplied by it)
        f = fmaxf(__uint_as_float((uint32_t)(127 - e) << 23) * a.scale_log2, FLT_MIN);
#pragma unroll 2
        for (int c = 0; c < kHalfChunks; ++c) {
          const uint32_t at = row + (((first + c) ^ (r & 7)) << 4);
          const uint4 u = dev::lds128(at);
          uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 y = dev::act2<F16>(x[i]);
            x[i] = dev::pack_act<true>(y.x * up, y.y * up);
          }
          sts128(at, x[0], x[1], x[2], x[3]);
        }
        fence_smem();
        __syncwarp();
        if (lane == 0 && ok) dev::mbar_arrive(dev::smem_u32(&q_full[t]));
        if (issuer && ok) {
          ok = all_wait(q_full[t], segs) && all_wait(k_full[it % kStages], it / kStages);
          fence_after();
          if (ok) scores(it);
        }
        ++segs;
      }
      // the earliest row of the tile sees everything up to here
      const int all_see = s.P + (int)((uint32_t)rho0 / (uint32_t)p.G);
      const int see = live ? s.P + tok : -1;
      float m_ref = -INFINITY, l = 0.f, sub = 0.f;   // (sub: the weights' exponent, 0 before the first reference)
      // the 64 weights of one half row under the present reference, and the
      // largest score; the S columns stay as they are
      auto weights = [&](int j, auto masked, uint32_t* pk, float& sum) {
        constexpr bool kMasked = decltype(masked)::value;
        const int seen = see - kKeys * j - 64 * h + 1;   // keys of the half that the row sees
        const float2 f2 = make_float2(f, f), neg = make_float2(-sub, -sub);
        float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        float mx[2] = {-INFINITY, -INFINITY};
        uint32_t v[2][8];
        ld8(s_addr, v[0]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t* x = v[c & 1];
          wait_ld();
          if (c < 7) ld8(s_addr + 8 * (c + 1), v[(c + 1) & 1]);
          if (kMasked) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (8 * c + k >= seen) x[k] = 0xff800000u;
          }
#pragma unroll
          for (int k = 0; k < 8; k += 4) {
            mx[0] = max3(mx[0], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
            mx[1] = max3(mx[1], __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
          }
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            float2 e = dev::fma2(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), f2, neg);
            e.x = ex2_approx(e.x);
            e.y = ex2_approx(e.y);
            part[(k >> 1) & 1] = dev::add2(part[(k >> 1) & 1], e);
            pk[4 * c + k / 2] = dev::pack_act<true>(e.x, e.y);
          }
        }
        part[0] = dev::add2(part[0], part[1]);
        sum = part[0].x + part[0].y;
        const float top = __fmul_ru(fmaxf(mx[0], mx[1]), f);
        return top < -kScoreMax ? -INFINITY : top;
      };
      for (int j = j0; j < j1; ++j) {
        if (ok) ok = all_wait(s_full[t], blocks);
        fence_after();
        // every row of the tile sees the block?
        const bool whole = kKeys * (j + 1) <= all_see + 1;
        uint32_t pk[32];
        float sum = 0.f, top = -INFINITY;
        for (;;) {
          if (ok) top = whole ? weights(j, std::false_type(), pk, sum) : weights(j, std::true_type(), pk, sum);
          // has a row's score passed its reference by more than 2^8?  (The first
          // block of a segment always does; the second vote on a block never.)
          if (!any_of(pair, 64, ok && top > __fadd_rd(m_ref, kLazyMax))) break;
          exchange[t][h][r] = top;
          named_sync(pair, 64);
          top = fmaxf(top, exchange[t][h ^ 1][r]);
          const float m_new = top > __fadd_rd(m_ref, kLazyMax) ? top : m_ref;
          const float sub_new = m_new == -INFINITY ? 0.f : __fadd_ru(m_new, -kHead);
          const float factor = m_new != m_ref && m_ref != -INFINITY ? ex2_approx(sub - sub_new) : 1.f;
          m_ref = m_new;
          sub = sub_new;
          l = m_new >= kScoreMax ? NAN : l * factor;
          if (ok && j > j0) {
            ok = all_wait(pv_done[t], blocks - 1);
            fence_after();
            if (ok) {
#pragma unroll 1
              for (int d = 0; d < D / 2; d += 16) {
                uint32_t x[16];
                ld16(o_addr + d, x);
                wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * factor);
                st16(o_addr + d, x);
              }
            }
          }
        }
        l += sum;
        if (ok) {
          st16(s_addr, pk);
          st16(s_addr + 16, pk + 16);
          wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0 && ok) dev::mbar_arrive(dev::smem_u32(&p_full[t]));
        if (issuer && ok) {
          ok = all_wait2(v_full[it % kStages], it / kStages, p_full[t], blocks);
          fence_after();
          if (ok) {
            const uint32_t vd = sw128_desc(v_base + (it % kStages) * C::kVTile);
#pragma unroll
            for (int m = 0; m < kTerms; ++m)
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_ts(el, tmem + o_col(t), tmem + s_col(t) + 64u * (kk >> 2) + 8u * (kk & 3),
                       vd + m * (C::kVTerm >> 4) + (kk >> 2) * (C::kVAtom >> 4) + 2 * (kk & 3), id_pv,
                       (j > j0 || m > 0 || kk > 0) ? 1u : 0u);
            commit(el, dev::smem_u32(&pv_done[t]));
            commit(el, dev::smem_u32(&v_empty[it % kStages]));
            if (j + 1 < j1) {
              // the next scores go over P, which this product still reads
              ok = all_wait2(k_full[(it + 1) % kStages], (it + 1) / kStages, pv_done[t], blocks);
              fence_after();
              if (ok) scores(it + 1);
            }
          }
        }
        ++blocks;
        ++it;
      }
      // the row's sum; O, divided by it where this CTA has the whole segment
      named_sync(pair, 64);   // (the last exchange has been read)
      exchange[t][h][r] = l;
      named_sync(pair, 64);
      l += exchange[t][h ^ 1][r];
      if (ok) ok = all_wait(pv_done[t], blocks - 1);
      fence_after();
      if (!ok) return true;
      const bool whole_seg = j0 == 0 && j1 == s.nb;
      const float inv = whole_seg ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const long long slot = ((long long)cta * 2 + (j0 == 0 ? 1 : 0)) * kPairRows + kTile * t;
      if (!whole_seg && h == 0)
        a.ml[slot + r] = live ? make_float2(m_ref == -INFINITY ? m_ref : sub, l) : make_float2(-INFINITY, 0.f);
      // 32 dims at a time through this warp's part of the Q tile (the last
      // scores are formed), so that stores to global memory are whole lines
      const uint32_t stage = q_tile + (uint32_t)(C::kQTile / 8) * (uint32_t)(warp & 7);
      constexpr int kCols = D / 4;               // dims of a pass: two passes for the thread's half
#pragma unroll 1
      for (int c = 0; c < D / 2; c += kCols) {
        uint32_t x[kCols];
        if (kCols == 32) ld32(o_addr + c, x);
        else ld16(o_addr + c, x);
        wait_ld();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kCols / 4; ++k)
          sts128(stage + r % 32 * (kCols * 4) + ((k ^ (r & (kCols / 4 - 1))) << 4),
                 __float_as_uint(__uint_as_float(x[4 * k]) * inv), __float_as_uint(__uint_as_float(x[4 * k + 1]) * inv),
                 __float_as_uint(__uint_as_float(x[4 * k + 2]) * inv),
                 __float_as_uint(__uint_as_float(x[4 * k + 3]) * inv));
        __syncwarp();
        constexpr int kLanes = kCols / 4;        // lanes of a row
#pragma unroll 1
        for (int i = 0; i < kLanes; ++i) {
          const int rr = 32 / kLanes * i + lane / kLanes, k = lane % kLanes;
          const int row = 32 * (warp & 3) + rr, rho2 = rho0 + row;
          const uint4 y = dev::lds128(stage + rr * (kCols * 4) + ((k ^ (rr & (kLanes - 1))) << 4));
          if (rho2 >= s.R) continue;
          const int dim = D / 2 * h + c + 4 * k;
          if (whole_seg) {
            const int tok2 = (int)((uint32_t)rho2 / (uint32_t)p.G);
            const long long o_row = (long long)(s.row0 + tok2) * p.Hq + s.kv * p.G + rho2 - tok2 * p.G;
            const float y0 = __uint_as_float(y.x), y1 = __uint_as_float(y.y), y2 = __uint_as_float(y.z),
                        y3 = __uint_as_float(y.w);
            const uint2 w = F16 || !a.out_f16 ? make_uint2(dev::pack_act<F16>(y0, y1), dev::pack_act<F16>(y2, y3))
                                              : make_uint2(dev::pack_act2(y0, y1, true), dev::pack_act2(y2, y3, true));
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o_row * D + dim) = w;
          } else {
            *reinterpret_cast<uint4*>(a.part + (slot + row) * D + dim) = y;
          }
        }
      }
      fence_before();   // (the next segment's products write O and S)
      return true;
    });
    if (issuer && !ok) {
      // a wait gave up: the products in flight end before their memory goes
      commit(el, dev::smem_u32(&drained[t]));
      dev::mbar_wait_until(dev::smem_u32(&drained[t]), 0, dev::globaltimer_ns() + kWaitLimitNs);
    }
  }
  if (!ok) *abort_v = 1;
  fence_before();
  __syncthreads();
  if (warp == kDecodeWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
  if (*abort_v) {
    describe(PageShared{});
    return;
  }

  // ---- the segment that goes on in the next CTA
  if (warp == 0) {
    PageShared x = {};
    Seg s = first_seg;
    int j = first_block;
    for (long long u = c0; u < c1;) {
      const int je = (int)min((long long)s.nb, j + (c1 - u));
      if (j == 0 && je < s.nb) {
        x.parts = owner(u + s.nb - 1) - cta + 1;
        x.row0 = s.row0;
        x.R = s.R;
        x.tile = s.tile;
        x.kv = s.kv;
      }
      u += je - j;
      j = 0;
      if (u < c1) advance(s);
    }
    describe(x);
  }
}

template <int D, bool F16>
cudaError_t setup_one() {
  return cudaFuncSetAttribute(page_attn_tc_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D, F16>::kSmem);
}

}  // namespace

cudaError_t page_attn_tc_setup() {
  cudaError_t e = setup_one<128, false>();
  if (e == cudaSuccess) e = setup_one<64, false>();
  if (e == cudaSuccess) e = setup_one<128, true>();
  if (e == cudaSuccess) e = setup_one<64, true>();
  return e;
}

cudaError_t launch_page_attn_tc(const PagesDev& p, const PageAttendTc& a, int ctas, cudaStream_t st) {
  if (p.d == 128)
    return p.f16 ? launch_k(page_attn_tc_kernel<128, true>, dim3(ctas), kThreads, Tc<128, true>::kSmem, st, p, a)
                 : launch_k(page_attn_tc_kernel<128, false>, dim3(ctas), kThreads, Tc<128, false>::kSmem, st, p, a);
  return p.f16 ? launch_k(page_attn_tc_kernel<64, true>, dim3(ctas), kThreads, Tc<64, true>::kSmem, st, p, a)
               : launch_k(page_attn_tc_kernel<64, false>, dim3(ctas), kThreads, Tc<64, false>::kSmem, st, p, a);
}

}  // namespace kvr
