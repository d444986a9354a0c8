// Attention over the 4-bit pages for sequences with many rows (kvr_page_attend):
// suffix prefill and wide speculative verify, on the 5th-generation tensor cores.
//
// S = Q K^T and O += P V in blocks of 128 keys, softmax in one pass with a lazy
// running maximum (a row's O is rescaled only when its maximum grows by more
// than 2^8).  K and V become fp16 tiles in shared memory: c - 8 exactly (as in
// k_page_attn.cu), times the scale, rounded once (2^-11; the product has at most
// 14 bits); q is scaled per row by a power of two so that any bf16 q is an fp16
// number; P is fp16 (2^-11).  Sums, maxima and O are fp32.
//
// Writing a 4-bit block as fp16 costs about as many instructions as the softmax
// of one 128-row tile over it, so a CTA runs two row tiles over each block: one
// dequantisation feeds four products.  Tensor memory holds S (P over it) and O
// of both tiles, 512 columns; while the softmax of one tile runs, the tensor
// core works for the other.  Warp roles (13 warps, four on a scheduler at most, so
// that a thread may hold 128 registers):
//   0-3, 4-7   softmax of tile 0 / 1, a thread per row: S from tensor memory 32
//              keys at a time, P back over the part of S already read; Q into
//              shared memory at the start of a segment
//   8-11       a quarter of each block's keys, global -> registers (one block
//              ahead) -> the fp16 tiles: K [128 keys][d] and V as [d][128 keys]
//              (both K-major with the 128-byte swizzle), two stages each
//   12         one thread issues the products
// The work, all (sequence, pair of row tiles, KV head, key block) units in this
// order, is cut into equal runs, one per CTA, whatever the lengths are; parts of
// a segment (one sequence, pair and head) that several CTAs hold are merged by
// the last of them to arrive, in the order of the keys.
//
// A NaN scale: of K, it makes the key's score NaN.  Of V, it would reach rows
// that do not see the key (0 * NaN), so the key's score becomes NaN instead and
// the value 0: rows that see it read NaN.
// Every wait is bounded; a CTA whose wait gave up frees its tensor memory.
#include <type_traits>

#include "kvr_pages.cuh"

namespace kvr {

namespace {

constexpr int kTile = 128;
constexpr int kPairRows = 2 * kTile;
constexpr int kKeys = 128;
constexpr int kDecodeWarp = 8, kMmaWarp = 12;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr float kLazyMax = 8.0f;

template <int D>
struct Tc {
  static constexpr int kGroups = D / 32;
  static constexpr int kQTile = kTile * D * 2;   // d / 64 atoms of [128 rows][64 dims]
  static constexpr int kQAtom = kTile * 128;
  static constexpr int kKTile = kKeys * D * 2;   // d / 64 atoms of [128 keys][64 dims]
  static constexpr int kKAtom = kKeys * 128;
  static constexpr int kVTile = D * kKeys * 2;   // 2 atoms of [d dims][64 keys]
  static constexpr int kVAtom = D * 128;
  static constexpr int kStages = 2;
  static constexpr int kSmem = 2 * kQTile + kStages * (kKTile + kVTile) + 1024;
  static constexpr int kSlot = kPairRows * D;    // floats of a partial result
};
// tensor memory columns
__device__ __forceinline__ uint32_t s_col(int t) { return (uint32_t)(128 * t); }
__device__ __forceinline__ uint32_t o_col(int t) { return (uint32_t)(256 + 128 * t); }

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// The product warp runs as one (every lane the same control flow, the elected
// lane's instructions predicated), so that the operands stay in uniform
// registers: from a branch of one lane each product cost about 117 cycles to
// issue instead of the 64 that it takes.
__device__ __forceinline__ uint32_t elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ void mma_ss(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t elected, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected)
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
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// two fp32 lanes in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
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
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  __half2 r = __hadd2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
// a number or, for NaN, 0 (scales are not negative)
__device__ __forceinline__ uint32_t number2(uint32_t s) {
  __half2 r = __hmax2(*reinterpret_cast<__half2*>(&s), __float2half2_rn(0.f));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t held(uint32_t x) {
  asm volatile("" : "+r"(x));
  return x;
}
// the four code pairs of a word as fp16 numbers c - 8, times s
struct Pairs {
  uint32_t v[4];
};
__device__ __forceinline__ Pairs decode(uint32_t w, uint32_t s, uint32_t k1024, uint32_t k64) {
  const uint32_t y = w >> 8;
  uint32_t a, b, c, d;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(a) : "r"(w), "r"(k1024));
  asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(b) : "r"(w), "r"(k64));
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(c) : "r"(y), "r"(k1024));
  asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(d) : "r"(y), "r"(k64));
  Pairs p;
  p.v[0] = hmul2(hadd2(a, 0xe408e408u), s);
  p.v[1] = hmul2(hadd2(b, 0xd480d480u), s);
  p.v[2] = hmul2(hadd2(c, 0xe408e408u), s);
  p.v[3] = hmul2(hadd2(d, 0xd480d480u), s);
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
  using C = Tc<D>;
  using K = Chunk<D>;
  constexpr int kG = C::kGroups;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full[2], s_full[2], p_full[2], pv_done[2], drained;
  __shared__ __align__(8) uint64_t k_full[C::kStages], k_empty[C::kStages], v_full[C::kStages], v_empty[C::kStages];
  __shared__ long long first_unit[kPageMaxSeqs + 1];   // units before each sequence
  __shared__ int start[4];                             // this CTA's first unit: sequence, tile, head, block
  __shared__ uint32_t tmem_slot;
  __shared__ int last_flag[2];
  __shared__ int abort_flag;
  volatile int* abort_v = &abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  const uint32_t base = (dev::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_base = base, k_base = q_base + 2 * C::kQTile, v_base = k_base + C::kStages * C::kKTile;

  dev::pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      dev::mbar_init(dev::smem_u32(&q_full[i]), 4);
      dev::mbar_init(dev::smem_u32(&s_full[i]), 1);
      dev::mbar_init(dev::smem_u32(&p_full[i]), 4);
      dev::mbar_init(dev::smem_u32(&pv_done[i]), 1);
    }
    dev::mbar_init(dev::smem_u32(&drained), 1);
    for (int i = 0; i < C::kStages; ++i) {
      dev::mbar_init(dev::smem_u32(&k_full[i]), 4);
      dev::mbar_init(dev::smem_u32(&k_empty[i]), 1);
      dev::mbar_init(dev::smem_u32(&v_full[i]), 4);
      dev::mbar_init(dev::smem_u32(&v_empty[i]), 1);
    }
    dev::fence_mbar_init();
  }
  dev::pdl_wait();
  if (tid == 0) *abort_v = dev::status_set(p.status) ? 1 : 0;

  // ---- units before every sequence: a warp per sequence sums its pairs' blocks
  const int n = p.info[0];
  const int rows_all = min(a.rows, p.info[1]);
  auto load_seq = [&](int b, Seg& s) {
    const int row0 = p.cu[b], row1 = p.cu[b + 1];
    s.b = b;
    s.row0 = row0;
    s.m = max(0, min(row1, rows_all) - row0);
    s.len = p.lens[b];
    s.P = s.len - (row1 - row0);
    s.R = p.G * s.m;
    return s.R > a.many;
  };
  auto blocks_of = [&](const Seg& s, int tile) {
    const int last = (int)((uint32_t)(min(s.R, kPairRows * (tile + 1)) - 1) / (uint32_t)p.G);
    return (s.P + last + kKeys) / kKeys;
  };
  for (int b = warp; b < n; b += kThreads / 32) {
    Seg s;
    long long u = 0;
    if (load_seq(b, s))
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
  if (units == 0 || *abort_v) return;
  const int ctas = (int)min((long long)gridDim.x, (units + a.min_units - 1) / a.min_units);
  if (cta >= ctas) return;
  const long long c0 = units * cta / ctas, c1 = units * (cta + 1) / ctas;
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
    s.kv = (int)(rem / s.nb);
    start[0] = s.b;
    start[1] = s.tile;
    start[2] = s.kv;
    start[3] = (int)(rem % s.nb);
  };
  if (warp == 0) locate(c0);
  if (warp == kMmaWarp) {
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
  auto all_wait = [&](uint64_t& bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
  auto slot_o = [&](int c, int i) { return a.part + ((long long)c * 2 + i) * C::kSlot; };
  auto slot_ml = [&](int c, int i) { return a.ml + ((long long)c * 2 + i) * kPairRows; };
  // 8 dims of an output row
  auto store8 = [&](const Seg& s, int rho, int d, const float* x) {
    const int tok = (int)((uint32_t)rho / (uint32_t)p.G);
    const long long row = (long long)(s.row0 + tok) * p.Hq + s.kv * p.G + rho - tok * p.G;
    uint4 v;
    if (F16 || !a.out_f16)
      v = make_uint4(dev::pack_act<F16>(x[0], x[1]), dev::pack_act<F16>(x[2], x[3]), dev::pack_act<F16>(x[4], x[5]),
                     dev::pack_act<F16>(x[6], x[7]));
    else
      v = make_uint4(dev::pack_act2(x[0], x[1], true), dev::pack_act2(x[2], x[3], true),
                     dev::pack_act2(x[4], x[5], true), dev::pack_act2(x[6], x[7], true));
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * D + d) = v;
  };

  bool ok = true;
  if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- products
    {
      const uint32_t el = elect();
      const uint32_t id_qk = idesc_f16(kTile, kKeys), id_pv = idesc_f16(kTile, D);
      uint32_t it = 0, segs[2] = {0, 0}, done[2] = {0, 0};   // blocks; segments and blocks of each tile
      auto scores = [&](int t, uint32_t i) {
        const uint64_t qd = sw128_desc(q_base + t * C::kQTile), kd = sw128_desc(k_base + (i & 1) * C::kKTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(el, tmem + s_col(t), qd + (kk >> 2) * (C::kQAtom >> 4) + 2 * (kk & 3),
                 kd + (kk >> 2) * (C::kKAtom >> 4) + 2 * (kk & 3), id_qk, kk > 0 ? 1u : 0u);
        commit(el, dev::smem_u32(&s_full[t]));
      };
      ok = for_segments([&](const Seg& s, int j0, int j1) {
        const int tiles = kPairRows * s.tile + kTile < s.R ? 2 : 1;
        if (!all_wait(k_full[it & 1], it >> 1)) return false;
        for (int t = 0; t < tiles; ++t) {
          if (!all_wait(q_full[t], segs[t]++)) return false;
          fence_after();
          scores(t, it);
        }
        commit(el, dev::smem_u32(&k_empty[it & 1]));
        for (int j = j0; j < j1; ++j, ++it) {
          const bool more = j + 1 < j1;
          for (int t = 0; t < tiles; ++t) {
            if (t == 0 && !all_wait(v_full[it & 1], it >> 1)) return false;
            if (!all_wait(p_full[t], done[t])) return false;
            fence_after();
            const uint64_t vd = sw128_desc(v_base + (it & 1) * C::kVTile);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma_ts(el, tmem + o_col(t), tmem + s_col(t) + 8u * (uint32_t)kk,
                     vd + (kk >> 2) * (C::kVAtom >> 4) + 2 * (kk & 3), id_pv, (j > j0 || kk > 0) ? 1u : 0u);
            commit(el, dev::smem_u32(&pv_done[t]));
            if (t + 1 == tiles) commit(el, dev::smem_u32(&v_empty[it & 1]));
            if (more) {
              // the next scores go over P, which this product still reads
              if (t == 0 && !all_wait(k_full[(it + 1) & 1], (it + 1) >> 1)) return false;
              if (!all_wait(pv_done[t], done[t])) return false;
              fence_after();
              scores(t, it + 1);
              if (t + 1 == tiles) commit(el, dev::smem_u32(&k_empty[(it + 1) & 1]));
            }
            ++done[t];
          }
        }
        return true;
      });
      if (!ok) {
        // a wait gave up: the products in flight end before their memory goes
        commit(el, dev::smem_u32(&drained));
        dev::mbar_wait_until(dev::smem_u32(&drained), 0, dev::globaltimer_ns() + kWaitLimitNs);
      }
    }
  } else if (warp >= kDecodeWarp) {
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
        if (it >= 2 && !all_wait(k_empty[it & 1], (it >> 1) - 1)) return false;
        const uint32_t k_tile = k_base + (it & 1) * C::kKTile;
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
            const Pairs x = decode(kc[i][jj], s2, k1024, k64);
            sts128(k_tile + (jj >> 1) * C::kKAtom + dev::swz128(key, 4 * (jj & 1) + t), x.v[0], x.v[1], x.v[2],
                   x.v[3]);
          }
        }
        fence_smem();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_u32(&k_full[it & 1]));
        if (j + 1 < j1) fetch_k(next_page);
        if (it >= 2 && !all_wait(v_empty[it & 1], (it >> 1) - 1)) return false;
        const uint32_t v_tile = v_base + (it & 1) * C::kVTile + (kb >> 3) * C::kVAtom;
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
          Pairs x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = decode(vc[i][jj], number2(vs[i][jj]), k1024, k64);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sts128(v_tile + dev::swz128(32 * jj + 4 * g + e, kbp), x[0].v[e], x[1].v[e], x[2].v[e], x[3].v[e]);
        }
        fence_smem();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_u32(&v_full[it & 1]));
        if (j + 1 < j1) {
          fetch_v(next_page);
          next_page = page_of(j + 2);
        }
      }
      return true;
    });
  } else {
    // ---------------------------------------------------------------- softmax
    const int t = warp >> 2;                   // row tile
    const int r = 32 * (warp & 3) + lane;      // row of it
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_addr = lanes + s_col(t), o_addr = lanes + o_col(t);
    uint32_t blocks = 0;                       // blocks of this tile so far
    ok = for_segments([&](const Seg& s, int j0, int j1) {
      const int rho0 = kPairRows * s.tile + kTile * t;
      if (rho0 >= s.R) return true;            // one tile only
      const int rho = rho0 + r;
      const bool live = rho < s.R;
      const int tok = live ? (int)((uint32_t)rho / (uint32_t)p.G) : 0;
      float f;
      {
        // q, scaled by a power of two with max|q| 2^e in [2^10, 2^11), as fp16
        const uint16_t* src =
            static_cast<const uint16_t*>(a.q) + (long long)(s.row0 + tok) * a.qs + (s.kv * p.G + rho - tok * p.G) * D;
        uint4 u[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          u[c] = make_uint4(0, 0, 0, 0);
          if (live) u[c] = *reinterpret_cast<const uint4*>(src + 8 * c);
        }
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t x[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 y = dev::act2<F16>(x[i]);
            top = max3(top, fabsf(y.x), fabsf(y.y));
          }
        }
        int e = 137 - (int)(__float_as_uint(top) >> 23);
        e = top > 0.f ? max(-100, min(100, e)) : 0;
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        f = __uint_as_float((uint32_t)(127 - e) << 23) * a.scale_log2;
        const uint32_t tile = q_base + t * C::kQTile;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t x[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 y = dev::act2<F16>(x[i]);
            x[i] = dev::pack_act<true>(y.x * up, y.y * up);
          }
          sts128(tile + (c >> 3) * C::kQAtom + dev::swz128(r, c & 7), x[0], x[1], x[2], x[3]);
        }
        fence_smem();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_u32(&q_full[t]));
      }
      // the earliest row of the tile sees everything up to here
      const int all_see = s.P + (int)((uint32_t)rho0 / (uint32_t)p.G);
      const int see = live ? s.P + tok : -1;
      float m_ref = -INFINITY, l = 0.f;
      float sub = 0.f;                         // the reference, 0 before the first
      float2 sum = make_float2(0.f, 0.f);
      // A row's score passed its reference by more than 2^8 in the part of the
      // block from key 32 c on: move the references, and what was formed under
      // them (O, the sums, the block's earlier weights) along.
      auto move_reference = [&](float top, int c, bool has_o) {
        const float m_new = top > m_ref + kLazyMax ? top : m_ref;
        const float factor = m_new != m_ref && m_ref != -INFINITY ? ex2_approx(m_ref - m_new) : 1.f;
        m_ref = m_new;
        sub = m_new == -INFINITY ? 0.f : m_new;
        l *= factor;
        sum.x *= factor;
        sum.y *= factor;
        if (has_o) {
          if (!all_wait(pv_done[t], blocks - 1)) return false;
          fence_after();
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            uint32_t x[16];
            ld16(o_addr + d, x);
            wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * factor);
            st16(o_addr + d, x);
          }
        }
        wait_st();   // (the weights stored so far are read back)
#pragma unroll 1
        for (int d = 0; d < c; ++d) {
          uint32_t x[16];
          ld16(s_addr + 16 * d, x);
          wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 y = dev::act2<true>(x[k]);
            x[k] = dev::pack_act<true>(y.x * factor, y.y * factor);
          }
          st16(s_addr + 16 * d, x);
        }
        return true;
      };
      auto block = [&](int j, auto masked) {
        constexpr bool kMasked = decltype(masked)::value;
        const int seen = see - kKeys * j + 1;   // keys of the block that the row sees
        const float2 f2 = make_float2(f, f);
        uint32_t v[2][32];
        ld32(s_addr, v[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t* x = v[c & 1];
          wait_ld();
          if (c < 3) ld32(s_addr + 32 * (c + 1), v[(c + 1) & 1]);
          if (kMasked) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (32 * c + k >= seen) x[k] = 0xff800000u;
          }
          float mx[2] = {__uint_as_float(x[0]), __uint_as_float(x[1])};
#pragma unroll
          for (int k = 2; k < 30; k += 4) {
            mx[0] = max3(mx[0], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
            mx[1] = max3(mx[1], __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
          }
          const float top = max3(mx[0], mx[1], fmaxf(__uint_as_float(x[30]), __uint_as_float(x[31]))) * f;
          if (__any_sync(0xffffffffu, top > m_ref + kLazyMax)) {
            wait_ld();   // (the loads of the slow path come after the one in flight)
            if (!move_reference(top, c, j > j0)) return false;
          }
          const float2 neg = make_float2(-sub, -sub);
          uint32_t pk[16];
          float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float2 e = fma2(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), f2, neg);
            e.x = ex2_approx(e.x);
            e.y = ex2_approx(e.y);
            part[(k >> 1) & 1] = add2(part[(k >> 1) & 1], e);
            pk[k / 2] = dev::pack_act<true>(e.x, e.y);
          }
          sum = add2(sum, add2(part[0], part[1]));
          st16(s_addr + 16 * c, pk);
        }
        wait_st();
        l += sum.x + sum.y;
        sum = make_float2(0.f, 0.f);
        return true;
      };
      for (int j = j0; j < j1; ++j) {
        if (!all_wait(s_full[t], blocks)) return false;
        fence_after();
        const bool whole = kKeys * (j + 1) <= all_see + 1;   // every row of the tile sees the block
        if (!(whole ? block(j, std::false_type()) : block(j, std::true_type()))) return false;
        fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_u32(&p_full[t]));
        ++blocks;
      }
      // O, divided by its sum where this CTA has the whole segment
      if (!all_wait(pv_done[t], blocks - 1)) return false;
      fence_after();
      const bool whole_seg = j0 == 0 && j1 == s.nb;
      const float inv = whole_seg ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const int slot = j0 == 0 ? 1 : 0;
      const int pr = kTile * t + r;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t x[32];
        ld32(o_addr + c, x);
        wait_ld();
        if (!live) continue;
        float y[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(x[k]) * inv;
        if (whole_seg) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) store8(s, rho, c + k, y + k);
        } else {
          float* dst = slot_o(cta, slot) + (long long)pr * D + c;
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<float4*>(dst + k) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
        }
      }
      if (!whole_seg) slot_ml(cta, slot)[pr] = live ? make_float2(m_ref, l) : make_float2(-INFINITY, 0.f);
      fence_before();   // (the next segment's products write O and S)
      return true;
    });
  }
  if (!ok) *abort_v = 1;
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
  if (*abort_v) return;

  // ---- segments shared with the CTAs before (0) and after (1)
  long long seg0[2] = {-1, -1};
  Seg seg[2];
  {
    Seg s = first_seg;
    int j = first_block;
    for (long long u = c0; u < c1;) {
      const int je = (int)min((long long)s.nb, j + (c1 - u));
      if (j > 0) {
        seg0[0] = u - j;
        seg[0] = s;
      } else if (je < s.nb) {
        seg0[1] = u;
        seg[1] = s;
      }
      u += je - j;
      j = 0;
      if (u < c1) advance(s);
    }
  }
  if (seg0[0] < 0 && seg0[1] < 0) return;
  auto owner = [&](long long u) { return (int)(((u + 1) * ctas - 1) / units); };
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      last_flag[i] = 0;
      if (seg0[i] < 0) continue;
      const int ca = owner(seg0[i]), cb = owner(seg0[i] + seg[i].nb - 1);
      if (dev::atom_add_acq_rel(a.counters + ca, 1) == cb - ca) {
        a.counters[ca] = 0;
        last_flag[i] = 1;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!last_flag[i]) continue;
    const Seg s = seg[i];
    const int ca = owner(seg0[i]), parts = owner(seg0[i] + s.nb - 1) - ca + 1;
    const int rows = min(kPairRows, s.R - kPairRows * s.tile);
    // a warp takes four rows at a time, a lane 4 (2) dims of each: the parts'
    // loads of all four are in flight together
    constexpr int kPer = D / 32;
    for (int r0 = 4 * warp; r0 < rows; r0 += 4 * (kThreads / 32)) {
      float m[4], l[4], x[4][kPer];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        m[q] = -INFINITY;
        l[q] = 0.f;
#pragma unroll
        for (int d = 0; d < kPer; ++d) x[q][d] = 0.f;
      }
#pragma unroll 2
      for (int k = 0; k < parts; ++k) {
        const float2* mls = slot_ml(ca + k, k == 0) + r0;
        const float* os = slot_o(ca + k, k == 0) + (long long)r0 * D + kPer * lane;
        float2 ml[4];
        float y[4][kPer];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          ml[q] = __ldcg(mls + q);   // (the slots have whole tiles of rows)
          if (kPer == 4) {
            const float4 z = __ldcg(reinterpret_cast<const float4*>(os + q * D));
            y[q][0] = z.x; y[q][1] = z.y; y[q][kPer - 2] = z.z; y[q][kPer - 1] = z.w;
          } else {
            const float2 z = __ldcg(reinterpret_cast<const float2*>(os + q * D));
            y[q][0] = z.x; y[q][1] = z.y;
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
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
      for (int q = 0; q < 4; ++q) {
        if (r0 + q >= rows) break;
        const float inv = l[q] == 0.f ? 0.f : 1.f / l[q];
        const int rho = kPairRows * s.tile + r0 + q;
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
}

template <int D, bool F16>
cudaError_t setup_one() {
  return cudaFuncSetAttribute(page_attn_tc_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::kSmem);
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
    return p.f16 ? launch_k(page_attn_tc_kernel<128, true>, dim3(ctas), kThreads, Tc<128>::kSmem, st, p, a)
                 : launch_k(page_attn_tc_kernel<128, false>, dim3(ctas), kThreads, Tc<128>::kSmem, st, p, a);
  return p.f16 ? launch_k(page_attn_tc_kernel<64, true>, dim3(ctas), kThreads, Tc<64>::kSmem, st, p, a)
               : launch_k(page_attn_tc_kernel<64, false>, dim3(ctas), kThreads, Tc<64>::kSmem, st, p, a);
}

}  // namespace kvr
