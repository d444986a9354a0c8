// Low-rank adapters beside a shared projection (include/kvr.h).
//
// Two launches, s = A x and out = base + scale B s: all outputs need all of s, and both
// read their matrices once.  s is held scaled by a row's power of two, in three terms of the type
// whose sum is s to 24 bits and more, so that B's products are those of 16-bit matrix units and s is held as
// a 32-bit float would hold it.
//
// Few rows a sequence.  shrink_kernel cuts the inputs into parts so that the CTAs
// fill the SMs whatever the rows are, and every part leaves its sums; expand_kernel
// adds the parts in their order, and B s to base.  Both walk tiles of eight rows, and
// in a tile the runs of rows that share an adapter: mma.sync takes the adapters'
// rows (16 of A or B) as its M side and the tile's as its N side.  Lanes load operands
// straight from global memory, 16 or 8 bytes each: which inputs share a fragment
// does not matter as long as both operands agree.  Bound: the chain of loads (whose rows, which
// adapter, where it is, its values), twice; where each row has its own adapter, the loads of A
// and B.  q, k and v of 3584 inputs, one row of rank 16: 8.0 us; of 4096 inputs, 64 rows with an
// adapter each: 18.1 us (40 MB).  Eight sequences of 8 rows, 18944 inputs, 32-bit outputs: 11.2 us.
//
// Many: tiles of one sequence's rows, below.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "kvr_batch.cuh"

namespace cg = cooperative_groups;

namespace kvr {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int R = kAdaptRows;
constexpr int kTileCols = 16 * kWarps;   // outputs of an expand CTA

template <class T>
__device__ __forceinline__ void mma(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// a pair of bf16 values held as fp16
__device__ __forceinline__ uint32_t bf16_of_half2(uint32_t v) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
  return dev::pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ float from(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float from(__half x) { return __half2float(x); }
template <class T>
__device__ __forceinline__ T to(float x) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// pairs of T
template <class T>
__device__ __forceinline__ float2 pair_from(uint32_t v) {
  if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&v));
  else return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <class T>
__device__ __forceinline__ uint32_t pair_to(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return dev::pack_bf16x2(lo, hi);
  }
}

// Terms of s: each leaves half a step of what the one before it left, 2^-8 for bf16, 2^-11 for fp16.  (With two,
// bf16 outputs of 254 rows were 1e-4 of their norm from those of s in 32-bit floats, and 0.5 us faster of 17.)
constexpr int kTerms = 3;

// What a row whose largest element is `big` is multiplied by to be held in terms of T (`down`, a power of two: to
// below 2, for fp16 to below 2^15, where elements far below the largest still have all their bits: their terms end
// at 2^-24), and its product with B in the end (`factor`, with the adapter's scale).  Neither leaves the normal
// numbers, whatever the row's and the scale's sizes are.  NaN in `down` for a row that is not finite.
template <class T>
__device__ __forceinline__ void scale_of(float big, float scale, float& down, float& factor) {
  constexpr int kTop = std::is_same<T, __half>::value ? 14 : 0;
  const int of_big = (int)(__float_as_uint(big) >> 23) - 127 - kTop;
  const int of_scale = (int)(__float_as_uint(fabsf(scale)) >> 23) - 127;
  const int e = min(max(of_big, max(-112, -125 - of_scale)), min(126, 126 - of_scale));
  down = big < INFINITY ? __int_as_float((127 - e) << 23) : __int_as_float(0x7fffffff);
  factor = scale * __int_as_float((e + 127) << 23);
}

// One output's B s, with s as it is.  (For sums that are NaN: an infinity in B times a term that is 0, or of the other
// sign than s, makes them so, where B s is infinite.)
template <class T>
__device__ __forceinline__ float one_sum(const T* b, const T* const (&terms)[kTerms], int rank) {
  float sum = from(terms[0][0]);
  if (sum != sum) return sum;   // (a row that is not finite: all of its terms are NaN)
  sum = 0.f;
  for (int j = 0; j < rank; ++j) {
    float s = 0.f;
#pragma unroll
    for (int m = kTerms - 1; m >= 0; --m) s += from(terms[m][j]);
    sum = fmaf(from(b[j]), s, sum);
  }
  return sum;
}

constexpr int kNone = -1;      // a row without an adapter
constexpr int kOutside = -2;   // a row of no sequence

// A tile's rows, their runs that share an adapter, and the runs' steps of 16 ranks.
struct Run {
  const void *a, *b;
  float scale;
  int rank, first, end;
};
struct Rows {
  int id[R];
  kvr_adapter ad[R];
  Run run[R];
  int runs, steps;
  uint8_t step_run[R * KVR_MAX_RANK * 3 / 16], step_j[R * KVR_MAX_RANK * 3 / 16];
};
// STEPS: the runs' steps are wanted, of the adapters' stacked ranks.
template <bool STEPS>
__device__ __forceinline__ void find_rows(const AdaptParams& p, int row0, int* cu, int* which, Rows& rows) {
  for (int i = threadIdx.x; i <= p.n_seq; i += kThreads) {
    cu[i] = p.cu[i];
    if (i < p.n_seq) which[i] = p.which[i];
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, r = row0 + lane;
    int id = kOutside;
    kvr_adapter e = {};
    if (lane < R) {
      int a = 0, b = p.n_seq + 1;   // first entry above r
      while (a < b) {
        const int m = (a + b) >> 1;
        if (cu[m] <= r) a = m + 1;
        else b = m;
      }
      if (r < p.rows && a > 0 && a <= p.n_seq) {
        id = which[a - 1];
        if (id < 0 || id >= p.site.n_adapters) id = kNone;
        if (id != kNone) {
          e = p.site.table[id];
          if (e.rank < 8 || e.rank > p.site.max_rank || e.rank % 8 || !e.a || !e.b) id = kNone;
        }
      }
      rows.id[lane] = id;
    }
    // runs: a row that differs from the one before starts one
    const int before = __shfl_up_sync(0xffffffffu, id, 1);
    const bool starts = lane < R && id >= 0 && (lane == 0 || before != id);
    const uint32_t all = __ballot_sync(0xffffffffu, starts), same = __ballot_sync(0xffffffffu, lane < R && id >= 0 && !starts);
    const int steps = STEPS && starts ? (e.rank * p.site.n_parts + 15) / 16 : 0;
    int at = steps;
#pragma unroll
    for (int o = 1; o < R; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += v;
    }
    if (starts) {
      const int k = __popc(all & ((1u << lane) - 1));
      const uint32_t after = ~(same >> (lane + 1));
      rows.run[k] = {e.a, e.b, e.scale, e.rank, lane, lane + __ffs(after)};
      for (int j = 0; j < steps; ++j) {
        rows.step_run[at - steps + j] = (uint8_t)k;
        rows.step_j[at - steps + j] = (uint8_t)j;
      }
    }
    at = __shfl_sync(0xffffffffu, at, R - 1);
    if (lane == 0) {
      rows.runs = __popc(all);
      rows.steps = at;
    }
  }
  __syncthreads();
}

// s = A x of one tile of rows and one part of the inputs: a warp takes 16 rows of A
// of a run at a time.  (So a row's sums are formed in one order, whatever shares its tile.)
template <class T>
__global__ void __launch_bounds__(kThreads) shrink_kernel(const AdaptParams p) {
  __shared__ int cu[kAdaptMaxSeqs + 1], which[kAdaptMaxSeqs];
  __shared__ Rows rows;
  dev::pdl_trigger();
  dev::pdl_wait();
  const int row0 = blockIdx.x * R, split = blockIdx.y;
  find_rows<true>(p, row0, cu, which, rows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int ld = p.site.n_parts * p.site.max_rank;
  const int K = p.site.k, chunks = (K + 31) / 32;
  const int c0 = (int)((long long)chunks * split / p.ksplit), c1 = (int)((long long)chunks * (split + 1) / p.ksplit);
  const uint4* xr = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + p.x_stride * (row0 + g));
  float* part = p.part + ((long long)split * p.rows + row0) * ld;
  for (int s = warp + kWarps * blockIdx.z; s < rows.steps; s += kWarps * gridDim.z) {
    const Run& run = rows.run[rows.step_run[s]];
    const int q = 16 * rows.step_j[s] + g, ranks = p.site.n_parts * run.rank;
    const bool in_run = g >= run.first && g < run.end;
    const T* lo_at = static_cast<const T*>(run.a) + (long long)q * K;
    const T* hi_at = lo_at + 8ll * K;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    // four chunks of 32 inputs in flight, and in one chain of products (which cut their sums, kChain)
    constexpr int kFlight = 4;
    for (int c = c0; c < c1; c += kFlight) {
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      uint4 xv[kFlight], lo[kFlight], hi[kFlight];
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int k = 32 * (c + f) + 8 * t;
        const bool in = c + f < c1 && k < K;
        lo[f] = in && q < ranks ? *reinterpret_cast<const uint4*>(lo_at + k) : zero;
        hi[f] = in && q + 8 < ranks ? *reinterpret_cast<const uint4*>(hi_at + k) : zero;
        xv[f] = in && in_run ? xr[k >> 3] : zero;
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        if (std::is_same<T, __nv_bfloat16>::value && p.x16) {
          xv[f].x = bf16_of_half2(xv[f].x);
          xv[f].y = bf16_of_half2(xv[f].y);
          xv[f].z = bf16_of_half2(xv[f].z);
          xv[f].w = bf16_of_half2(xv[f].w);
        }
        mma<T>(acc, lo[f].x, hi[f].x, lo[f].y, hi[f].y, xv[f].x, xv[f].y);
        mma<T>(acc, lo[f].z, hi[f].z, lo[f].w, hi[f].w, xv[f].z, xv[f].w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += acc[e];
    }
    // rows q and q + 8 of A, rows 2 t and 2 t + 1 of x
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 2 * t + (e & 1), j = q + 8 * (e >> 1);
      if (r >= run.first && r < run.end && j < ranks) part[(long long)r * ld + j] = sum[e];
    }
  }
}

// out = base + scale B s of one tile of rows and 16 outputs a warp.
template <class T, class O>
__global__ void __launch_bounds__(kThreads, 2) expand_kernel(const AdaptParams p) {
  constexpr int kS = KVR_MAX_RANK + 8;   // (rows shifted against one another in the banks)
  __shared__ int cu[kAdaptMaxSeqs + 1], which[kAdaptMaxSeqs];
  __shared__ Rows rows;
  __shared__ __align__(16) T terms[kTerms][R][kS];
  __shared__ float factor[R];
  __shared__ __align__(16) float tile[R][kTileCols + 4];
  dev::pdl_trigger();
  dev::pdl_wait();
  const int row0 = blockIdx.x * R;
  find_rows<false>(p, row0, cu, which, rows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // the CTA's part, its outputs' place in it and in out
  int part = 0, col = blockIdx.y, left = 0;
  for (;; ++part) {
    const int tiles = (p.site.cols[part] + kTileCols - 1) / kTileCols;
    if (col < tiles) break;
    col -= tiles;
    left += p.site.cols[part];
  }
  col *= kTileCols;
  const int cols = min(kTileCols, p.site.cols[part] - col);
  const int ld = p.site.n_parts * p.site.max_rank;

  // A warp takes a run, or a share of its outputs where there are fewer runs than
  // warps.  Its first B, and base, are on their way while s is added up.
  const int share = rows.runs > 4 ? 1 : rows.runs > 2 ? 2 : rows.runs > 1 ? 4 : 8;   // warps of a run
  const int mine = warp / share;
  const Run run = rows.run[mine < rows.runs ? mine : 0];
  const int tiles = mine < rows.runs ? kWarps / share : 0, tile0 = warp % share * (kWarps / share);
  const T* B = static_cast<const T*>(run.b) + (long long)(left + col + 16 * tile0 + g) * run.rank + 4 * t;
  uint2 lo[kWarps], hi[kWarps];
  auto fetch = [&](int j0) {
#pragma unroll
    for (int n = 0; n < kWarps; ++n) {
      lo[n] = hi[n] = make_uint2(0u, 0u);
      const int c = 16 * (tile0 + n) + g;
      const bool in = n < tiles && j0 + 4 * t < run.rank;
      if (in && c < cols) lo[n] = *reinterpret_cast<const uint2*>(B + (long long)(16 * n) * run.rank + j0);
      if (in && c + 8 < cols) hi[n] = *reinterpret_cast<const uint2*>(B + (long long)(16 * n + 8) * run.rank + j0);
    }
  };
  fetch(0);
  const int r = warp, i = 4 * lane;   // (the row and the outputs that this lane writes)
  const int id = rows.id[r];
  const long long at = left + col + i;
  const bool writes = id != kOutside && i < cols && !(id == kNone && p.base == p.out);
  O* out = static_cast<O*>(p.out) + p.out_stride * (row0 + r) + at;
  const O* base = p.base && writes ? static_cast<const O*>(p.base) + p.base_stride * (row0 + r) + at : nullptr;
  float4 base_f = make_float4(0.f, 0.f, 0.f, 0.f);
  uint2 base_h = make_uint2(0u, 0u);
  if (base) {
    if constexpr (std::is_same<O, float>::value) base_f = *reinterpret_cast<const float4*>(base);
    else base_h = *reinterpret_cast<const uint2*>(base);
  }

  // s of row `warp`: the parts' sum, scaled by a power of two to below 2, in terms of T
  if (id >= 0) {
    int k = 0;
    while (r >= rows.run[k].end) ++k;
    const int rank = rows.run[k].rank;
    const int plane = p.rows * ld;   // (below 2^31: what few rows a sequence and 2048 sequences make)
    float v[KVR_MAX_RANK / 32], big = 0.f;
#pragma unroll
    for (int n = 0; n < KVR_MAX_RANK / 32; ++n) {
      const int j = lane + 32 * n;
      v[n] = 0.f;
      if (j < rank) {
        const float* src = p.part + (long long)(row0 + r) * ld + part * rank + j;
        int s = 0;
        for (; s + 8 <= p.ksplit; s += 8, src += 8ll * plane) {
          float w[8];
#pragma unroll
          for (int k2 = 0; k2 < 8; ++k2) w[k2] = src[k2 * (long long)plane];
#pragma unroll
          for (int k2 = 0; k2 < 8; ++k2) v[n] += w[k2];
        }
        for (; s < p.ksplit; ++s, src += plane) v[n] += *src;
      }
      big = fmaxf(big, fabsf(v[n]));
      if (v[n] != v[n]) big = INFINITY;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    float down;
    float f;
    scale_of<T>(big, rows.run[k].scale, down, f);
#pragma unroll
    for (int n = 0; n < KVR_MAX_RANK / 32; ++n) {
      const int j = lane + 32 * n;
      float x = v[n] * down;
      if (j < (rank + 15) / 16 * 16)
#pragma unroll
        for (int m = 0; m < kTerms; ++m) {
          const T h = to<T>(x);
          terms[m][r][j] = h;
          x -= from(h);
        }
    }
    if (lane == 0) factor[r] = f;
  }
  __syncthreads();
  if (tiles) {
    float acc[kWarps][4];
#pragma unroll
    for (int n = 0; n < kWarps; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    const bool in_run = g >= run.first && g < run.end;
    for (int j0 = 0; j0 < run.rank; j0 += 16) {
      if (j0) fetch(j0);
      uint2 y[kTerms];
#pragma unroll
      for (int m = 0; m < kTerms; ++m)
        y[m] = in_run ? *reinterpret_cast<const uint2*>(&terms[m][g][j0 + 4 * t]) : make_uint2(0u, 0u);
#pragma unroll
      for (int n = 0; n < kWarps; ++n)
        if (n < tiles)
#pragma unroll
          for (int m = kTerms - 1; m >= 0; --m) mma<T>(acc[n], lo[n].x, hi[n].x, lo[n].y, hi[n].y, y[m].x, y[m].y);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 2 * t + e;
      if (row < run.first || row >= run.end) continue;
      const float f = factor[row];
#pragma unroll
      for (int n = 0; n < kWarps; ++n)
        if (n < tiles) {
          tile[row][16 * (tile0 + n) + g] = acc[n][e] * f;
          tile[row][16 * (tile0 + n) + g + 8] = acc[n][2 + e] * f;
        }
    }
  }
  __syncthreads();
  if (!writes) return;
  float4 v = id >= 0 ? *reinterpret_cast<const float4*>(&tile[r][i]) : make_float4(0.f, 0.f, 0.f, 0.f);
  if (v.x != v.x || v.y != v.y || v.z != v.z || v.w != v.w) {
    int k = 0;
    while (r >= rows.run[k].end) ++k;
    const int rank = rows.run[k].rank;
    const T* const row[kTerms] = {terms[0][r], terms[1][r], terms[2][r]};
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      const float y = c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w;
      if (y == y) continue;
      const float z = one_sum(static_cast<const T*>(rows.run[k].b) + (at + c) * rank, row, rank) * factor[r];
      if (c == 0) v.x = z;
      else if (c == 1) v.y = z;
      else if (c == 2) v.z = z;
      else v.w = z;
    }
  }
  if constexpr (std::is_same<O, float>::value) {
    if (id >= 0) {   // (else base's own bits)
      base_f.x += v.x;
      base_f.y += v.y;
      base_f.z += v.z;
      base_f.w += v.w;
    }
    *reinterpret_cast<float4*>(out) = base_f;
  } else {
    __align__(8) O w[4];
    *reinterpret_cast<uint2*>(w) = base_h;
    if (id >= 0) {
      w[0] = to<O>(from(w[0]) + v.x);
      w[1] = to<O>(from(w[1]) + v.y);
      w[2] = to<O>(from(w[2]) + v.z);
      w[3] = to<O>(from(w[3]) + v.w);
    }
    *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(w);
  }
}

// ---------------------------------------------------------------- many rows a sequence
// Tiles of one sequence's rows.  shrink_tiles_kernel streams 64 rows of x and A through
// shared memory (a cluster cuts the inputs, its CTAs' sums are joined in distributed
// shared memory) and leaves s in terms of T, by tcgen05 or mma.sync (launch_tiles); expand_tiles_kernel
// multiplies 128 rows of them with 128 outputs' B while base is on its way, on tcgen05.
// Addresses are the adapters', known on the device only, so copies are cp.async, not tensor maps'.
// Bound: shrink by what it moves from L2 to the SMs (each 64 inputs of 64 rows bring up to 192 rows
// of A; 64 rows of x instead of 128, since two CTAs an SM cover each other's start and end),
// expand by base and out.  Four ragged prompts, 6.7k rows of 4096 inputs, rank 64, 6144 outputs:
// 91 us, of which a plain copy of x, base and out would take 33; with 32-bit base and out 117 of 57.
constexpr int TR = 64;
constexpr int kStep = 64;       // inputs of a stage: 128 bytes a row
constexpr int kStages = 3;      // (4 and 6 leave one CTA an SM for 192 rows of A: four prompts 103 us, with 3 91)
constexpr int kMaxCluster = 8;
constexpr int ER = 128, kTileN = 128;   // rows and outputs of a tile of expand

__host__ __device__ inline int round16(int r) { return (r + 15) & ~15; }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  const int bytes = valid ? 16 : 0;   // (0: zeros, nothing is read)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct Tile {
  int tiles;           // of the batch
  int row0, rows;      // 0 rows: none
  int id;              // adapter, or kNone
  kvr_adapter ad;
};
// Tile `t` of the batch: sequences in order, each in tiles of ROWS rows.
template <int ROWS>
__device__ __forceinline__ void find_tile(const AdaptParams& p, int t, Tile& tile) {
  __shared__ int warp_sum[kWarps];
  constexpr int kPer = kAdaptMaxSeqs / kThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.n_seq + kThreads - 1) / kThreads;   // sequences a thread, 1 .. kPer
  const int b0 = threadIdx.x * per;
  if (threadIdx.x == 0) tile.rows = 0;
  int n[kPer], sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    n[k] = 0;
    if (k < per && b0 + k < p.n_seq) {
      const int r0 = max(p.cu[b0 + k], 0), r1 = min(p.cu[b0 + k + 1], p.rows);
      n[k] = r1 > r0 ? (r1 - r0 + ROWS - 1) / ROWS : 0;
    }
    sum += n[k];
  }
  int run = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
  }
  if (lane == 31) warp_sum[warp] = run;
  __syncthreads();
  int at = run - sum;
  for (int k = 0; k < warp; ++k) at += warp_sum[k];
  if (threadIdx.x == kThreads - 1) tile.tiles = at + sum;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (t >= at && t < at + n[k]) {
      const int b = b0 + k;
      const int r0 = max(p.cu[b], 0), r1 = min(p.cu[b + 1], p.rows);
      tile.row0 = r0 + (t - at) * ROWS;
      tile.rows = min(r1 - tile.row0, ROWS);
      int id = p.which[b];
      if (id < 0 || id >= p.site.n_adapters) id = kNone;
      if (id != kNone) {
        const kvr_adapter e = p.site.table[id];
        if (e.rank < 8 || e.rank > p.site.max_rank || e.rank % 8 || !e.a || !e.b) id = kNone;
        tile.ad = e;
      }
      tile.id = id;
    }
    at += n[k];
  }
  __syncthreads();
}

// The low-rank products of the tiles: terms [k][row][part * round16(max_rank)] and
// a factor for each row and part, behind one another in p.part.
struct Terms {
  int ld, rows;
  uint8_t* base;
  __host__ __device__ explicit Terms(const AdaptParams& p)
      : ld(p.site.n_parts * round16(p.site.max_rank)), rows(p.rows), base(reinterpret_cast<uint8_t*>(p.part)) {}
  template <class T>
  __device__ __forceinline__ T* term(int k, int row) const {
    return reinterpret_cast<T*>(base) + ((long long)k * rows + row) * ld;
  }
  __device__ __forceinline__ float* factor(int row) const {
    return reinterpret_cast<float*>(base + (long long)kTerms * rows * ld * 2) + row * 3;
  }
  __host__ __device__ size_t bytes() const { return (size_t)kTerms * rows * ld * 2 + (size_t)rows * 12; }
};

// The tensor memory's products: operands in shared memory, rows of 128 bytes in the 128-byte swizzle,
// eight of them 1024 bytes apart; sums of row i of 128 in lane i.
__device__ __forceinline__ uint64_t smem_operand(uint32_t at) {
  return (uint64_t)((at >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
template <class T>
__device__ __forceinline__ constexpr uint32_t product_of(int m, int n) {
  constexpr uint32_t kType = std::is_same<T, __half>::value ? 0u : 1u;
  return (1u << 4) | (kType << 7) | (kType << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void tc_mma(uint32_t sums, uint64_t a, uint64_t b, uint32_t what, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(sums),
      "l"(a), "l"(b), "r"(what), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 32 columns of 16 lanes, as mma.sync's sums of four products lie in a warp.  (Products of 64 rows have sixteen of them
// in each 32 lanes.)
__device__ __forceinline__ void tc_load16x32(uint32_t at, float (&v)[4][4]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k / 4][k % 4] = __uint_as_float(r[k]);
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// One chunk of NC stacked rows of A (all parts, or one) of one tile and one part of the inputs.
// X16: x is fp16 that holds bf16 values.  TC: on tcgen05.
// Matrix units cut a sum's last bits at every product of 16 inputs instead of rounding them; over 4096 inputs in one
// chain that is 2e-6 of the sum.  So chains are kChain stages, added up in registers: below 3e-7.
constexpr int kChain = 2;
// (Three CTAs an SM where shared memory allows them: three parts of rank 128, 8192 rows, 115 us, with two 133; one part 80, 78.)
template <class T, int NC, bool TC, bool X16>
__global__ void __launch_bounds__(kThreads, TC && NC == 128 ? 3 : 2) shrink_tiles_kernel(const AdaptParams p, int ks) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ Tile tile;
  __shared__ __align__(8) uint64_t bars[kStages];   // of a stage's products
  __shared__ uint32_t sums_slot;
  constexpr int kSumCols = NC <= 128 ? 128 : 256;   // (TC)
  constexpr int kXBytes = TR * 128, kStage = kXBytes + NC * 128;
  constexpr int kNT = NC / 32;    // tiles of 8 ranks a warp
  constexpr int kLd = NC + 4;
  static_assert(TR * kLd * 4 <= kStages * kStage, "the sums fit where the stages were");
  uint8_t* smem = smem_raw + ((1024u - (dev::smem_u32(smem_raw) & 1023u)) & 1023u);
  if (!TC) dev::pdl_trigger();
  dev::pdl_wait();
  const int part_k = blockIdx.x % ks;
  find_tile<TR>(p, blockIdx.x / ks, tile);
  if (tile.rows == 0 || tile.id == kNone) return;   // (the whole cluster)
  const int rank = tile.ad.rank;
  const bool whole = gridDim.z == 1;
  const int q0 = whole ? 0 : blockIdx.z * rank, nq = whole ? p.site.n_parts * rank : rank;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = warp & 1, wn = warp >> 1;
  uint32_t sums_at = 0;
  if (TC) {
    if (warp == 0) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dev::smem_u32(&sums_slot)),
                   "r"(kSumCols));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else if (threadIdx.x == 32) {
#pragma unroll
      for (int i = 0; i < kStages; ++i) dev::mbar_init(dev::smem_u32(&bars[i]), 1);
      dev::fence_mbar_init();
    }
    tc_before();
    __syncthreads();
    tc_after();
    sums_at = sums_slot;
    // (only now: a kernel behind that takes tensor memory and waits for this one must not take it first)
    dev::pdl_trigger();
  }
  const int K = p.site.k, steps = (K + kStep - 1) / kStep;
  const int s0 = (int)((long long)steps * part_k / ks), s1 = (int)((long long)steps * (part_k + 1) / ks);
  const uint32_t base = dev::smem_u32(smem);
  // a thread copies 16 bytes of every 32nd row: where from and where to moves with the stage only
  constexpr int kRowStep = kThreads / 8;
  const int lr = threadIdx.x >> 3, lc = threadIdx.x & 7;
  const uint32_t to_smem = base + dev::swz128(lr, lc);
  const T* x = static_cast<const T*>(p.x) + p.x_stride * (tile.row0 + lr) + 8 * lc;
  const T* A = static_cast<const T*>(tile.ad.a) + (long long)(q0 + lr) * K + 8 * lc;
  const long long x_step = p.x_stride * kRowStep, a_step = (long long)K * kRowStep;
  const int x_rows = tile.rows - lr, a_rows = nq - lr;
  auto load = [&](int s, int at) {
    const uint32_t st = to_smem + at * kStage;
    const int k = s * kStep;
    const bool in = k + 8 * lc < K;
#pragma unroll
    for (int j = 0; j < TR / kRowStep; ++j) {
      const bool v = in && j * kRowStep < x_rows;
      cp16(st + j * kRowStep * 128, v ? x + j * x_step + k : p.x, v);
    }
#pragma unroll
    for (int j = 0; j < NC / kRowStep; ++j) {
      const bool v = in && j * kRowStep < a_rows;
      cp16(st + kXBytes + j * kRowStep * 128, v ? A + j * a_step + k : tile.ad.a, v);
    }
  };
  // a lane's 16-byte chunks of its operand rows, by the 16 inputs of a product
  uint32_t a_at[kStep / 16], b_at[kStep / 16];
#pragma unroll
  for (int kk = 0; kk < kStep / 16; ++kk) {
    a_at[kk] = base + dev::swz128(wr * 32 + (lane & 15), 2 * kk + (lane >> 4));
    b_at[kk] = base + kXBytes + dev::swz128(wn * (NC / 4) + (lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1));
  }
  // the chains' sums: TC: rows 16 (warp % 4) + g and + 8, outputs (warp / 4) NC / 2 + 8 n + 2 t and + 1
  constexpr int kSums = TC ? NC / 16 : 2 * kNT;
  float sum[kSums][4];
#pragma unroll
  for (int n = 0; n < kSums; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[n][e] = 0.f;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (s0 + i < s1) load(s0 + i, i);
    cp_commit();
  }
  int at = 0;
  // A wait that gives up ends the CTA's copies and products; its rows read NaN.
  bool ok = true;
  int issued = 0;   // steps whose products the first thread has issued
  // products of step s are over
  const auto over = [&](int s) {
    ok = ok && dev::mbar_wait(dev::smem_u32(&bars[(s - s0) % kStages]), (uint32_t)((s - s0) / kStages) & 1u, p.status);
  };
  if constexpr (TC) {
    for (int s = s0; s < s1; ++s) {
      cp_wait<kStages - 2>();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
      if (threadIdx.x == 0 && ok) {
        const uint32_t st = base + at * kStage;
        const uint64_t xd = smem_operand(st), ad = smem_operand(st + kXBytes);
        tc_after();
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          tc_mma(sums_at, xd + 2 * kk, ad + 2 * kk, product_of<T>(TR, NC), (s - s0) % kChain != 0 || kk > 0);
        tc_commit(dev::smem_u32(&bars[at]));
        ++issued;
      }
      // the stage of the step before, once its products are over
      if (s + kStages - 1 < s1) {
        if (s > s0) over(s - 1);
        if (ok) load(s + kStages - 1, at == 0 ? kStages - 1 : at - 1);
      }
      cp_commit();
      at = at + 1 == kStages ? 0 : at + 1;
      if ((s - s0) % kChain == kChain - 1 || s + 1 == s1) {   // (the next chain's products wait for every warp's loads)
        over(s);
        tc_after();
#pragma unroll
        for (int c = 0; c < kSums; c += 4) {
          float v[4][4];
          tc_load16x32(sums_at + ((uint32_t)(32 * (warp & 3)) << 16) + (warp >> 2) * (NC / 2) + 8 * c, v);
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[c + n][e] += v[n][e];
        }
        tc_before();
      }
    }
  } else {
    float acc[2][kNT][4];
    for (int s = s0; s < s1; ++s) {
      cp_wait<kStages - 2>();
      __syncthreads();
      if (s + kStages - 1 < s1) load(s + kStages - 1, at == 0 ? kStages - 1 : at - 1);
      cp_commit();
      const uint32_t st = at * kStage;
      at = at + 1 == kStages ? 0 : at + 1;
      if ((s - s0) % kChain == 0)
#pragma unroll
        for (int n = 0; n < kSums; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (s > s0) sum[n][e] += acc[n / kNT][n % kNT][e];
            acc[n / kNT][n % kNT][e] = 0.f;
          }
#pragma unroll
      for (int kk = 0; kk < kStep / 16; ++kk) {
        uint32_t a[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          dev::ldmatrix_x4(a_at[kk] + st + m * 16 * 128, a[m][0], a[m][1], a[m][2], a[m][3]);
          if (X16)
#pragma unroll
            for (int e = 0; e < 4; ++e) a[m][e] = bf16_of_half2(a[m][e]);
        }
#pragma unroll
        for (int n = 0; n < kNT; n += 2) {
          uint32_t b[4];   // ranks 8 n .. + 15: (first eight, low and high inputs), (second eight, ...)
          dev::ldmatrix_x4(b_at[kk] + st + n * 8 * 128, b[0], b[1], b[2], b[3]);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma<T>(acc[m][n], a[m][0], a[m][1], a[m][2], a[m][3], b[0], b[1]);
            mma<T>(acc[m][n + 1], a[m][0], a[m][1], a[m][2], a[m][3], b[2], b[3]);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kSums; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[n][e] += acc[n / kNT][n % kNT][e];
  }
  cp_wait<0>();
  if constexpr (TC) {
    ok = __syncthreads_and(ok);
    if (!ok) {   // (what is still under way reads the stages and writes the sums)
      if (issued)
        dev::mbar_wait_until(dev::smem_u32(&bars[(issued - 1) % kStages]), (uint32_t)((issued - 1) / kStages) & 1u,
                             dev::globaltimer_ns() + kWaitLimitNs);
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  // the cluster's sums, a share of the rows each, a warp a row
  float* sums = reinterpret_cast<float*>(smem);
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < kSums; ++n) {
    const int r = TC ? 16 * (warp & 3) + g : wr * 32 + n / kNT * 16 + g;
    const int q = TC ? (warp >> 2) * (NC / 2) + 8 * n : wn * (NC / 4) + n % kNT * 8;
    float* d = sums + r * kLd + q + 2 * t;
    if (!ok) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = __int_as_float(0x7fffffff);
    *reinterpret_cast<float2*>(d) = make_float2(sum[n][0], sum[n][1]);
    *reinterpret_cast<float2*>(d + 8 * kLd) = make_float2(sum[n][2], sum[n][3]);
  }
  if (TC && warp == 0) {   // (all warps' loads are over: the barrier above)
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sums_at), "r"(kSumCols));
  }
  const cg::cluster_group cluster = cg::this_cluster();
  if (ks > 1) cluster.sync();
  else __syncthreads();
  const int r0 = TR * part_k / ks, r1 = TR * (part_k + 1) / ks;
  if (ks > 1) {
    // the cluster's sums of this CTA's rows, in the order of the inputs: four at a
    // time, all CTAs' on their way together
    float4 sum[TR * NC / 4 / 2 / kThreads];   // (at most half of the rows)
    constexpr int kQuads = NC / 4;
#pragma unroll 1
    for (int i = threadIdx.x, n = 0; i < (r1 - r0) * kQuads; i += kThreads, ++n) {
      const int at = (r0 + i / kQuads) * kLd + i % kQuads * 4;
      float4 v[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        v[c] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(sums, c < ks ? c : 0) + at);
      float4 t = v[0];
#pragma unroll
      for (int c = 1; c < kMaxCluster; ++c)
        if (c < ks) {
          t.x += v[c].x;
          t.y += v[c].y;
          t.z += v[c].z;
          t.w += v[c].w;
        }
#pragma unroll
      for (int k = 0; k < (int)(sizeof(sum) / sizeof(float4)); ++k)
        if (k == n) sum[k] = t;
    }
    cluster.sync();   // (everyone has read them)
#pragma unroll
    for (int n = 0; n < (int)(sizeof(sum) / sizeof(float4)); ++n) {
      const int i = threadIdx.x + n * kThreads;
      if (i < (r1 - r0) * kQuads)
        *reinterpret_cast<float4*>(sums + (r0 + i / kQuads) * kLd + i % kQuads * 4) = sum[n];
    }
    __syncthreads();
  }
  const Terms terms(p);
  const int parts = whole ? p.site.n_parts : 1, mr16 = round16(p.site.max_rank);
  for (int i = r0 * parts + warp; i < min(r1, tile.rows) * parts; i += kWarps) {
    const int r = i / parts, j = i % parts;
    float v[KVR_MAX_RANK / 32], big = 0.f;
#pragma unroll
    for (int n = 0; n < KVR_MAX_RANK / 32; ++n) {
      const int q = lane + 32 * n;
      v[n] = q < rank ? sums[r * kLd + j * rank + q] : 0.f;
      big = fmaxf(big, fabsf(v[n]));
      if (v[n] != v[n]) big = INFINITY;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    float down;
    float factor;
    scale_of<T>(big, tile.ad.scale, down, factor);
    const int pj = whole ? j : blockIdx.z;
#pragma unroll
    for (int k = 0; k < kTerms; ++k) {
      T* dst = terms.term<T>(k, tile.row0 + r) + pj * mr16;
#pragma unroll
      for (int n = 0; n < KVR_MAX_RANK / 32; ++n) {
        const int q = lane + 32 * n;
        if (q < round16(rank)) {
          const float y = k == 0 ? v[n] * down : v[n];
          const T h = to<T>(y);
          dst[q] = h;
          v[n] = y - from(h);
        }
      }
    }
    if (lane == 0) terms.factor(tile.row0 + r)[pj] = factor;
  }
}

// Eight outputs of a row: base's, and what is added to them.
template <class O>
struct Eight {
  uint4 v[sizeof(O) / 2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < (int)sizeof(O) / 2; ++k) v[k] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void load(const O* p) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(O) / 2; ++k) v[k] = reinterpret_cast<const uint4*>(p)[k];
  }
  __device__ __forceinline__ void store(O* p) const {
#pragma unroll
    for (int k = 0; k < (int)sizeof(O) / 2; ++k) reinterpret_cast<uint4*>(p)[k] = v[k];
  }
  // pair k += (y0, y1) f
  __device__ __forceinline__ void add(int k, float y0, float y1, float f) {
    uint32_t* w = reinterpret_cast<uint32_t*>(v);
    if constexpr (std::is_same<O, float>::value) {
      w[2 * k] = __float_as_uint(fmaf(y0, f, __uint_as_float(w[2 * k])));
      w[2 * k + 1] = __float_as_uint(fmaf(y1, f, __uint_as_float(w[2 * k + 1])));
    } else {
      const float2 b = pair_from<O>(w[k]);
      w[k] = pair_to<O>(fmaf(y0, f, b.x), fmaf(y1, f, b.y));
    }
  }
};

// A warp's outputs of a tile one by one, where some of its sums are not finite: those that are NaN are formed anew
// (one_sum).  `sums` and `b`: of the warp's and the lane's first output `col` of the part.
template <class T, class O>
__device__ __noinline__ void outputs_one_by_one(const AdaptParams& p, const Tile& tile, const float* factor, uint32_t sums,
                                                const T* b, int part, int left, int col, int c_end, int row0) {
  const Terms terms(p);
  const int rank = tile.ad.rank;
  for (int m = 0; m < 2; ++m)
    for (int h = 0; h < 2; ++h) {
      float acc[4][4];
      tc_load16x32(sums + ((uint32_t)(16 * m) << 16) + 32 * h, acc);
      if (col + 32 * h >= c_end) continue;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int r = row0 + 16 * m + 8 * (k >> 1 & 1), n = 32 * h + 2 * (k >> 2) + (k & 1);
        if (r >= tile.rows) continue;
        const long long row = tile.row0 + r, at = left + col + n;
        float y = acc[k / 4][k % 4];
        if (y != y) {
          const T* s[kTerms];
#pragma unroll
          for (int j = 0; j < kTerms; ++j) s[j] = terms.term<T>(j, tile.row0 + r) + part * round16(p.site.max_rank);
          y = one_sum(b + (long long)n * rank, s, rank);
        }
        O* out = static_cast<O*>(p.out) + p.out_stride * row + at;
        const O* base = static_cast<const O*>(p.base) + p.base_stride * row + at;
        if constexpr (std::is_same<O, float>::value) *out = fmaf(y, factor[r], p.base ? *base : 0.f);
        else *out = to<O>(fmaf(y, factor[r], p.base ? from(*base) : 0.f));
      }
    }
}

// What a CTA keeps from run to run: its tensor memory (two tiles' sums), and their barriers' phases.
struct Sums {
  uint32_t at, bars;   // (bars: 8 bytes a tile)
  uint32_t phases;     // (a bit a tile)
  uint32_t issued;     // products that have not been waited for (the first thread's, a bit a tile)
  bool ok;             // no wait has given up: then no more copies and products, and outputs read NaN
};
constexpr int kOperand = ER * 128;   // bytes of 128 rows of 64 ranks

// `c1 - c0` tiles of 128 outputs of one part, of a tile of rows.  The outputs that
// stand beside one another in a lane's sums are chosen: its four pairs are eight in
// a row, so base and out need no way through shared memory.
template <class T, class O>
__device__ __forceinline__ void expand_run(const AdaptParams& p, const Tile& tile, float* factor, uint32_t smem, Sums& sums,
                                           int part, int left, int c0, int c1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int c_end = min(c1 * kTileN, p.site.cols[part]), n = c1 - c0;
  if (tile.id == kNone && p.base == p.out) return;
  const bool adapted = tile.id != kNone;
  const int rank = adapted ? tile.ad.rank : 0, r16 = round16(rank);
  const int halves = (round16(p.site.max_rank) + 63) / 64;   // operands of 64 ranks
  const uint32_t b_smem = smem + kTerms * halves * kOperand;
  // a thread's 16 bytes of a row of ranks (a power of two of them, the last ones without work)
  const int chunks = r16 / 8, shift = chunks > 1 ? 32 - __clz(chunks - 1) : 0;
  const int lr = threadIdx.x >> shift, lc = threadIdx.x & ((1 << shift) - 1), lstep = kThreads >> shift;
  const uint32_t half = (lc >> 3) * kOperand;
  // a lane's rows row0, + 8, + 16, + 24 and its outputs ocol .. + 7 and 32 further
  const int row0 = (warp & 3) * 32 + g, ocol = (warp >> 2) * 64 + 8 * t;
  const O* base = p.base ? static_cast<const O*>(p.base) + p.base_stride * (tile.row0 + row0) + left + ocol : nullptr;
  O* out = static_cast<O*>(p.out) + p.out_stride * (tile.row0 + row0) + left + ocol;
  const long long base8 = 8 * p.base_stride, out8 = 8 * p.out_stride;
  const auto fetch = [&](int col, Eight<O> (&o)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (base && col + ocol < c_end && row0 + 8 * k < tile.rows) o[k].load(base + col + k * base8);
      else o[k].clear();
    }
  };
  const auto store = [&](int col, const Eight<O> (&o)[4]) {
    if (col + ocol >= c_end) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (row0 + 8 * k < tile.rows) o[k].store(out + col + k * out8);
  };
  if (!adapted) {
    for (int col = c0 * kTileN; col < c_end; col += kTileN) {
      Eight<O> o[2][4];
      fetch(col, o[0]);
      fetch(col + 32, o[1]);
      store(col, o[0]);
      store(col + 32, o[1]);
    }
    return;
  }
  const T* B = static_cast<const T*>(tile.ad.b) + (long long)left * rank;
  const auto load = [&](int col, int buf) {
    if (lc < chunks && sums.ok) {
      const T* src = B + (long long)(col + lr) * rank + 8 * lc;
      const int step = lstep * rank;
      const uint32_t dst = b_smem + buf * halves * kOperand + half;
      const bool in = 8 * lc < rank;
      // output 8 t + 2 n + e of 32 is row 8 n + 2 t + e
#pragma unroll 4
      for (int r = lr; r < kTileN; r += lstep) {
        const bool v = in && col + r < c_end;
        cp16(dst + dev::swz128((r & ~31) | (r & 6) << 2 | (r & 24) >> 2 | (r & 1), lc & 7), v ? src : B, v);
        src += step;
      }
    }
    cp_commit();
  };
  // what the threads have copied, for the products: of buffer b into its sums
  const auto multiply = [&](int b) {
    cp_wait<0>();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_before();
    sums.ok = __syncthreads_and(sums.ok);
    if (threadIdx.x == 0 && sums.ok) {
      tc_after();
      const uint64_t bd = smem_operand(b_smem + b * halves * kOperand);
#pragma unroll 1
      for (int k = kTerms - 1; k >= 0; --k) {   // (the smallest terms first)
        const uint64_t sd = smem_operand(smem + k * halves * kOperand);
        for (int kk = 0; kk < r16 / 16; ++kk) {
          const int at = (kk >> 2) * (kOperand >> 4) + 2 * (kk & 3);
          tc_mma(sums.at + b * kTileN, sd + at, bd + at, product_of<T>(ER, kTileN), k < kTerms - 1 || kk > 0);
        }
      }
      tc_commit(sums.bars + 8 * b);
      sums.issued |= 1u << b;
    }
  };
  tc_before();
  sums.ok = __syncthreads_and(sums.ok);   // (the last run's factors have been read)
  if (sums.ok) {
    const Terms terms(p);
#pragma unroll
    for (int k = 0; k < kTerms; ++k)
      for (int r = lr; r < ER && lc < chunks; r += lstep) {
        const T* src = terms.term<T>(k, tile.row0 + min(r, tile.rows - 1)) + part * round16(p.site.max_rank) + 8 * lc;
        cp16(smem + k * halves * kOperand + half + dev::swz128(r, lc & 7), src, r < tile.rows);
      }
    if (threadIdx.x < tile.rows) factor[threadIdx.x] = terms.factor(tile.row0 + threadIdx.x)[part];
  }
  load(c0 * kTileN, 0);
  multiply(0);
  if (n > 1) load((c0 + 1) * kTileN, 1);
  for (int i = 0; i < n; ++i) {
    const int b = i & 1, col = (c0 + i) * kTileN;
    Eight<O> o[2][4];
    fetch(col, o[0]);
    fetch(col + 32, o[1]);
    if (i + 1 < n) multiply(b ^ 1);   // (its sums have been read: the last tile but one's)
    if (sums.ok && dev::mbar_wait(sums.bars + 8 * b, (sums.phases >> b) & 1u, p.status)) {
      sums.phases ^= 1u << b;
      sums.issued &= ~(1u << b);
    } else {
      sums.ok = false;
    }
    const bool ok = sums.ok = __all_sync(0xffffffffu, sums.ok);
    tc_after();
    if (i + 2 < n) load(col + 2 * kTileN, b);
    float z = 0.f;   // (NaN if a sum is not finite)
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float acc[4][4];
        tc_load16x32(sums.at + ((uint32_t)((warp & 3) * 32 + 16 * m) << 16) + b * kTileN + (warp >> 2) * 64 + 32 * h, acc);
#pragma unroll
        for (int k = 0; k < 16; ++k) z = fmaf(acc[k / 4][k % 4], 0.f, z);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float f = ok ? factor[row0 + 16 * m + 8 * k] : __int_as_float(0x7fffffff);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[h][2 * m + k].add(j, acc[j][2 * k], acc[j][2 * k + 1], f);
        }
      }
    if (ok && __any_sync(0xffffffffu, z != z)) {
      outputs_one_by_one<T, O>(p, tile, factor, sums.at + ((uint32_t)((warp & 3) * 32) << 16) + b * kTileN + (warp >> 2) * 64,
                               B + (long long)(col + ocol) * rank, part, left, col + ocol, c_end, row0);
      continue;
    }
    store(col, o[0]);
    store(col + 32, o[1]);
  }
}

// The tiles of 128 rows times their tiles of 128 outputs in equal runs, one a CTA:
// while 128 rows and a part last the terms stay, and the next outputs' products run
// and B is on its way while some are added to base and stored.
template <class T, class O>
__global__ void __launch_bounds__(kThreads, 2) expand_tiles_kernel(const AdaptParams p, int col_tiles) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ Tile tile;
  __shared__ float factor[ER];
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ uint32_t sums_slot;
  const uint32_t smem = (dev::smem_u32(smem_raw) + 1023u) & ~1023u;
  dev::pdl_wait();
  Sums sums = {0, dev::smem_u32(bars), 0, 0, true};
  if (threadIdx.x < 32) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dev::smem_u32(&sums_slot)),
                 "r"(2 * kTileN));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else if (threadIdx.x == 32) {
    dev::mbar_init(sums.bars, 1);
    dev::mbar_init(sums.bars + 8, 1);
    dev::fence_mbar_init();
  }
  tc_before();
  __syncthreads();
  tc_after();
  sums.at = sums_slot;
  dev::pdl_trigger();   // (only now: see shrink_tiles_kernel)
  find_tile<ER>(p, 0, tile);
  // (no more tiles than sequences in their order can have)
  const int units = min(tile.tiles, p.rows / ER + min(p.n_seq, p.rows)) * col_tiles;
  int u = (int)((long long)units * blockIdx.x / gridDim.x);
  const int u1 = (int)((long long)units * (blockIdx.x + 1) / gridDim.x);
  int now = 0;
  while (u < u1) {
    if (u / col_tiles != now) {
      now = u / col_tiles;
      __syncthreads();   // (the last one has been read)
      find_tile<ER>(p, now, tile);
    }
    const int first = u % col_tiles, n = min(u1 - u, col_tiles - first);
    int part = 0, before = 0, left = 0, tiles = 0;
    for (;; ++part) {
      tiles = (p.site.cols[part] + kTileN - 1) / kTileN;
      if (first < before + tiles) break;
      before += tiles;
      left += p.site.cols[part];
    }
    const int c0 = first - before, c1 = min(c0 + n, tiles);   // of this part
    u += c1 - c0;
    expand_run<T, O>(p, tile, factor, smem, sums, part, left, c0, c1);
  }
  tc_before();
  cp_wait<0>();
  if (!__syncthreads_and(sums.ok)) {   // (what is still under way reads the operands and writes the sums)
    for (int b = 0; b < 2; ++b)
      if (sums.issued >> b & 1)
        dev::mbar_wait_until(sums.bars + 8 * b, (sums.phases >> b) & 1u, dev::globaltimer_ns() + kWaitLimitNs);
    __syncthreads();
  }
  if (threadIdx.x < 32) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sums.at), "r"(2 * kTileN));
  }
}

int expand_tiles_smem(int max_rank) {
  return (round16(max_rank) + 63) / 64 * (kTerms + 2) * kOperand + 1024;   // (operands start where their swizzle does)
}
template <int NC>
constexpr int shrink_tiles_smem() {
  return kStages * (TR + NC) * 128 + 1024;   // (stages start where their swizzle does)
}

template <class T, int NC, bool TC>
cudaError_t launch_shrink_tiles(const AdaptParams& p, int tiles, int chunks, int sms, cudaStream_t st) {
  // CTAs of a tile: as many as two an SM (they run at a time), with 256 inputs each at least.  2048 rows of 18944
  // inputs, rank 32: 53 us, with up to 3/2 an SM 75; four prompts 91 either way, with up to 3 an SM 95.
  int ks = 1;
  while (ks < kMaxCluster && tiles * chunks * ks * 2 <= 2 * sms && p.site.k >= 512 * ks) ks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * ks), 1, (unsigned)chunks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = shrink_tiles_smem<NC>();
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)ks, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  if constexpr (std::is_same<T, __nv_bfloat16>::value && !TC)
    if (p.x16) return cudaLaunchKernelEx(&cfg, shrink_tiles_kernel<T, NC, TC, true>, p, ks);
  return cudaLaunchKernelEx(&cfg, shrink_tiles_kernel<T, NC, TC, false>, p, ks);
}

template <class T, class O>
cudaError_t launch_tiles(const AdaptParams& p, int sms, cudaStream_t st) {
  const int tiles = p.rows / TR + std::min(p.n_seq, p.rows);   // at most
  const int wide = p.rows / ER + std::min(p.n_seq, p.rows);
  const int stacked = p.site.n_parts * p.site.max_rank;
  // All parts at once, as far as a CTA's sums hold them.  On tcgen05 sums have to be fetched at the end of every chain:
  // products with 64 of A are too small for that, and 32-bit outputs are faster without.  Us, mma.sync and
  // tcgen05 (8192 rows): one output of 4096 inputs, rank 64, 60, 73; three of 3584, rank 64, 102, 84; four
  // prompts with 32-bit outputs (4096 inputs, three of rank 64) 117, 132.
  constexpr bool kTc = !std::is_same<O, float>::value;
  cudaError_t e;
  if (stacked <= 64) e = launch_shrink_tiles<T, 64, false>(p, tiles, 1, sms, st);
  else if (stacked <= 128) e = launch_shrink_tiles<T, 128, kTc>(p, tiles, 1, sms, st);
  else if (kTc && stacked <= 192) e = launch_shrink_tiles<T, kTc ? 192 : 128, kTc>(p, tiles, 1, sms, st);
  else if (p.site.max_rank <= 64) e = launch_shrink_tiles<T, 64, false>(p, tiles, p.site.n_parts, sms, st);
  else e = launch_shrink_tiles<T, 128, kTc>(p, tiles, p.site.n_parts, sms, st);
  if (e != cudaSuccess) return e;
  int cols = 0;
  for (int j = 0; j < p.site.n_parts; ++j) cols += (p.site.cols[j] + kTileN - 1) / kTileN;
  const int smem = expand_tiles_smem(p.site.max_rank);
  const int per_sm = smem <= 110 * 1024 ? 2 : 1;
  const int ctas = (int)std::min<long long>((long long)sms * per_sm, (long long)wide * cols);
  return launch_k(expand_tiles_kernel<T, O>, dim3(ctas), dim3(kThreads), smem, st, p, cols);
}

template <class T, int NC, bool TC, bool X16>
cudaError_t setup_shrink() {
  return cudaFuncSetAttribute(shrink_tiles_kernel<T, NC, TC, X16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              shrink_tiles_smem<NC>());
}
template <class T, class O>
cudaError_t setup_expand() {
  return cudaFuncSetAttribute(expand_tiles_kernel<T, O>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              expand_tiles_smem(KVR_MAX_RANK));
}

template <class T>
cudaError_t launch(const AdaptParams& p, cudaStream_t st) {
  const int blocks = (p.rows + R - 1) / R;
  // CTAs of a tile's part: enough that a warp has one step, if all sequences are alike and differ in
  // their adapters
  const int runs = std::min(R, (R * p.n_seq + p.rows - 1) / p.rows);
  const int steps = runs * ((p.site.n_parts * p.site.max_rank + 15) / 16);
  const dim3 shrink_grid(blocks, p.ksplit, std::min((steps + kWarps - 1) / kWarps, 4));
  cudaError_t e = launch_k(shrink_kernel<T>, shrink_grid, dim3(kThreads), 0, st, p);
  if (e != cudaSuccess) return e;
  int tiles = 0;
  for (int j = 0; j < p.site.n_parts; ++j) tiles += (p.site.cols[j] + kTileCols - 1) / kTileCols;
  const dim3 grid(blocks, tiles);
  if (p.out_type != KVR_ACT_F32) return launch_k(expand_kernel<T, T>, grid, kThreads, 0, st, p);
  return launch_k(expand_kernel<T, float>, grid, kThreads, 0, st, p);
}

// Rows of a sequence, on average, and in all, from which tiles of one sequence's rows pay.  Sequences x rows (all of one
// length), tiles of eight against these, us (q, k and v of 3584 inputs; rank 16): 32 x 8 20, 24; 32 x 16 34, 31; 64 x 16 67,
// 47; 8 x 8 9, 15; 8 x 16 13, 15 (rank 64: 19, 20); 8 x 24 16, 16; 1 x 40 9, 13.  One rule for a batch is not the best
// where lengths are unequal: 2048 rows and 150 single ones (14.6 on average) take 226 us, and 120 (17.9) 85.
constexpr int kManyRows = 16, kManyInAll = 128;

int adapt_split(const kvr_adapter_site& s, int rows, int sms) {
  // parts of the inputs: two CTAs an SM (8 x 8 rows of 18944 inputs: 11.2 us, one 13.1), of 192 inputs each at least
  // (64 rows of 4096 inputs, an adapter each: 18.1 us, with 128 19.6; one row: 8.0 and 7.4)
  const int blocks = (rows + R - 1) / R;
  const int most = std::max(1, std::min(kAdaptMaxSplit, s.k / 192));
  return std::max(1, std::min(most, 2 * sms / blocks));
}

}  // namespace

cudaError_t adapt_setup() {
  cudaError_t e = setup_shrink<__nv_bfloat16, 64, false, false>();
  if (e == cudaSuccess) e = setup_shrink<__nv_bfloat16, 128, false, false>();
  if (e == cudaSuccess) e = setup_shrink<__nv_bfloat16, 64, false, true>();   // (the layer stack's: 32-bit outputs)
  if (e == cudaSuccess) e = setup_shrink<__nv_bfloat16, 128, false, true>();
  if (e == cudaSuccess) e = setup_shrink<__nv_bfloat16, 128, true, false>();
  if (e == cudaSuccess) e = setup_shrink<__nv_bfloat16, 192, true, false>();
  if (e == cudaSuccess) e = setup_shrink<__half, 64, false, false>();
  if (e == cudaSuccess) e = setup_shrink<__half, 128, false, false>();
  if (e == cudaSuccess) e = setup_shrink<__half, 128, true, false>();
  if (e == cudaSuccess) e = setup_shrink<__half, 192, true, false>();
  if (e == cudaSuccess) e = setup_expand<__nv_bfloat16, __nv_bfloat16>();
  if (e == cudaSuccess) e = setup_expand<__nv_bfloat16, float>();
  if (e == cudaSuccess) e = setup_expand<__half, __half>();
  if (e == cudaSuccess) e = setup_expand<__half, float>();
  return e;
}

__device__ int g_gave_up;   // non-zero once a wait of a call without a context's status word has given up

cudaError_t adapt_status(int** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_gave_up); }

size_t adapt_work_bytes(const kvr_adapter_site& s, int rows) {
  // (of any number of SMs, for few or many rows a sequence)
  AdaptParams p = {};
  p.site = s;
  p.rows = rows;
  return std::max((size_t)adapt_split(s, rows, 1024) * rows * s.n_parts * s.max_rank * sizeof(float),
                  Terms(p).bytes());
}

cudaError_t launch_adapt(AdaptParams p, int sms, cudaStream_t st) {
  if (p.rows >= kManyInAll && p.rows >= kManyRows * (long long)p.n_seq) {
    if (p.site.type == KVR_ACT_F16)
      return p.out_type == KVR_ACT_F32 ? launch_tiles<__half, float>(p, sms, st) : launch_tiles<__half, __half>(p, sms, st);
    return p.out_type == KVR_ACT_F32 ? launch_tiles<__nv_bfloat16, float>(p, sms, st)
                                     : launch_tiles<__nv_bfloat16, __nv_bfloat16>(p, sms, st);
  }
  p.ksplit = adapt_split(p.site, p.rows, std::min(sms, 1024));
  return p.site.type == KVR_ACT_F16 ? launch<__half>(p, st) : launch<__nv_bfloat16>(p, st);
}

}  // namespace kvr
