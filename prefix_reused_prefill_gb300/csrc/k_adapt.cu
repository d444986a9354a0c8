// Low-rank adapters beside a shared projection (include/kvr.h).
//
// Two launches.  shrink_kernel forms s = A x: the inputs are cut into parts so that
// the CTAs fill the SMs whatever the rows are, and every part leaves its sums.
// expand_kernel adds the parts in their order, and B s to base.  Both walk tiles
// of consecutive rows, and in a tile the runs of rows that share an adapter.
//
// The tensor cores take the adapters' rows (16 of A or B) as their M side and
// rows of x or s as their N side.  Lanes load operands straight from global
// memory, 16 or 8 bytes each: which inputs share a fragment does not matter as
// long as both operands agree.
#include <algorithm>
#include <type_traits>

#include "kvr_batch.cuh"

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

constexpr int kNone = -1;      // a row without an adapter
constexpr int kOutside = -2;   // a row of no sequence

// The tile's rows: the adapter of each, and its entry.
struct Rows {
  int id[R];
  kvr_adapter ad[R];
};
__device__ __forceinline__ void find_rows(const AdaptParams& p, int row0, int* cu, Rows& rows) {
  for (int i = threadIdx.x; i <= p.n_seq; i += kThreads) cu[i] = p.cu[i];
  __syncthreads();
  if (threadIdx.x < R) {
    const int r = row0 + threadIdx.x;
    int a = 0, b = p.n_seq + 1;   // first entry above r
    while (a < b) {
      const int m = (a + b) >> 1;
      if (cu[m] <= r) a = m + 1;
      else b = m;
    }
    int id = kOutside;
    if (r < p.rows && a > 0 && a <= p.n_seq) {
      id = p.which[a - 1];
      if (id < 0 || id >= p.site.n_adapters) id = kNone;
      if (id != kNone) {
        const kvr_adapter e = p.site.table[id];
        if (e.rank < 8 || e.rank > p.site.max_rank || e.rank % 8 || !e.a || !e.b) id = kNone;
        rows.ad[threadIdx.x] = e;
      }
    }
    rows.id[threadIdx.x] = id;
  }
  __syncthreads();
}
// the next run [first, at) of rows that share an adapter; false behind the last one
__device__ __forceinline__ bool next_run(const Rows& rows, int& at, int& first) {
  while (at < R && rows.id[at] < 0) ++at;
  if (at == R) return false;
  first = at;
  while (at < R && rows.id[at] == rows.id[first]) ++at;
  return true;
}

// s = A x of one tile of rows and one part of the inputs.  A warp takes a run, or
// a share of its inputs where there are fewer runs than warps.
constexpr int kRankTiles = 4;   // 16 rows of A each, in registers at a time
template <class T>
__global__ void __launch_bounds__(kThreads) shrink_kernel(const AdaptParams p) {
  __shared__ int cu[kAdaptMaxSeqs + 1];
  __shared__ Rows rows;
  __shared__ float red[kWarps][kRankTiles][16 * R];
  dev::pdl_trigger();
  dev::pdl_wait();
  const int row0 = blockIdx.x * R, split = blockIdx.y;
  find_rows(p, row0, cu, rows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int ld = p.site.n_parts * p.site.max_rank;
  int runs = 0, most = 0;
  for (int at = 0, f; next_run(rows, at, f); ++runs) most = max(most, rows.ad[f].rank);
  if (runs == 0) return;
  const int per_run = kWarps / runs, sub = warp % per_run;
  int first = 0, end = 0, at = 0;
  const bool mine = warp / per_run < runs;
  for (int k = 0; mine && k <= warp / per_run; ++k) {
    next_run(rows, at, first);
    end = at;
  }
  const int K = p.site.k, chunks = (K + 31) / 32;
  const int c0 = (int)((long long)chunks * split / p.ksplit), c1 = (int)((long long)chunks * (split + 1) / p.ksplit);
  const int ranks = mine ? p.site.n_parts * rows.ad[first].rank : 0;
  const T* A = mine ? static_cast<const T*>(rows.ad[first].a) : nullptr;
  const bool in_run = mine && g >= first && g < end;
  const uint4* xr = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + p.x_stride * (row0 + g));
  float* part = p.part + ((long long)split * p.rows + row0) * ld;
  for (int j0 = 0; j0 < p.site.n_parts * most; j0 += 16 * kRankTiles) {
    float acc[kRankTiles][4];
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    if (j0 < ranks) {
#pragma unroll 2
      for (int c = c0 + sub; c < c1; c += per_run) {
        const int k = 32 * c + 8 * t;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        uint4 xv = in_run && k < K ? xr[k >> 3] : zero;
        uint4 lo[kRankTiles], hi[kRankTiles];
#pragma unroll
        for (int j = 0; j < kRankTiles; ++j) {
          const int q = j0 + 16 * j + g;
          lo[j] = q < ranks && k < K ? *reinterpret_cast<const uint4*>(A + (long long)q * K + k) : zero;
          hi[j] = q + 8 < ranks && k < K ? *reinterpret_cast<const uint4*>(A + (long long)(q + 8) * K + k) : zero;
        }
        if (std::is_same<T, __nv_bfloat16>::value && p.x16) {
          xv.x = bf16_of_half2(xv.x);
          xv.y = bf16_of_half2(xv.y);
          xv.z = bf16_of_half2(xv.z);
          xv.w = bf16_of_half2(xv.w);
        }
#pragma unroll
        for (int j = 0; j < kRankTiles; ++j) {
          if (j0 + 16 * j >= ranks) break;
          mma<T>(acc[j], lo[j].x, hi[j].x, lo[j].y, hi[j].y, xv.x, xv.y);
          mma<T>(acc[j], lo[j].z, hi[j].z, lo[j].w, hi[j].w, xv.z, xv.w);
        }
      }
    }
    // acc[j]: rows j0 + 16 j + g (and + 8) of A, rows 2 t and 2 t + 1 of x
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[warp][j][(2 * t + (e & 1)) * 16 + g + 8 * (e >> 1)] = acc[j][e];
    __syncthreads();
    if (mine && sub == 0) {
      for (int i = lane; i < kRankTiles * 16 * (end - first); i += 32) {
        const int q = i % (16 * kRankTiles), r = first + i / (16 * kRankTiles);
        if (j0 + q >= ranks) continue;
        float v = 0.f;
        for (int w = 0; w < per_run; ++w) v += red[warp + w][q >> 4][r * 16 + (q & 15)];
        part[(long long)r * ld + j0 + q] = v;
      }
    }
  }
}

// out = base + scale B s of one tile of rows and 16 outputs a warp.
template <class T, class O, int TERMS>
__global__ void __launch_bounds__(kThreads) expand_kernel(const AdaptParams p) {
  constexpr int kS = KVR_MAX_RANK + 8;   // (rows shifted against one another in the banks)
  __shared__ int cu[kAdaptMaxSeqs + 1];
  __shared__ Rows rows;
  __shared__ __align__(16) T terms[TERMS][R][kS];
  __shared__ float factor[R];
  __shared__ __align__(16) float tile[R][kTileCols + 4];
  dev::pdl_trigger();
  dev::pdl_wait();
  const int row0 = blockIdx.x * R;
  find_rows(p, row0, cu, rows);
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

  // s of row `warp`: the parts' sum, scaled by a power of two to below 2, in terms of T
  {
    const int r = warp;
    if (rows.id[r] >= 0) {
      const int rank = rows.ad[r].rank;
      const float* src = p.part + (long long)(row0 + r) * ld + part * rank;
      float v[KVR_MAX_RANK / 32], big = 0.f;
#pragma unroll
      for (int i = 0; i < KVR_MAX_RANK / 32; ++i) {
        const int j = lane + 32 * i;
        v[i] = 0.f;
        if (j < rank)
          for (int s = 0; s < p.ksplit; ++s) v[i] += src[(long long)s * p.rows * ld + j];
        big = fmaxf(big, fabsf(v[i]));
        if (v[i] != v[i]) big = INFINITY;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      // (a row that is not finite is NaN as a whole)
      const int e = min(max((int)(__float_as_uint(big) >> 23), 27), 253) - 127;
      const float down = big < INFINITY ? __int_as_float((127 - e) << 23) : __int_as_float(0x7fffffff);
#pragma unroll
      for (int i = 0; i < KVR_MAX_RANK / 32; ++i) {
        const int j = lane + 32 * i;
        float x = v[i] * down;
        if (j < (rank + 15) / 16 * 16)
#pragma unroll
          for (int k = 0; k < TERMS; ++k) {
            const T h = to<T>(x);
            terms[k][r][j] = h;
            x -= from(h);
          }
      }
      if (lane == 0) factor[r] = rows.ad[r].scale * __int_as_float((e + 127) << 23);
    }
  }
  __syncthreads();
  const int c = 16 * warp + g;
  for (int at = 0, first; next_run(rows, at, first);) {
    const int rank = rows.ad[first].rank;
    const T* B = static_cast<const T*>(rows.ad[first].b) + (long long)(left + col) * rank;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const bool in_run = g >= first && g < at;
#pragma unroll 2
    for (int j0 = 0; j0 < rank; j0 += 16) {
      const int j = j0 + 4 * t;
      const uint2 zero = make_uint2(0u, 0u);
      const uint2 lo = j < rank && c < cols ? *reinterpret_cast<const uint2*>(B + (long long)c * rank + j) : zero;
      const uint2 hi = j < rank && c + 8 < cols ? *reinterpret_cast<const uint2*>(B + (long long)(c + 8) * rank + j) : zero;
#pragma unroll
      for (int k = TERMS - 1; k >= 0; --k) {
        const uint2 s = in_run ? *reinterpret_cast<const uint2*>(&terms[k][g][j]) : zero;
        mma<T>(acc, lo.x, hi.x, lo.y, hi.y, s.x, s.y);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 2 * t + (e & 1);
      if (r >= first && r < at) tile[r][c + 8 * (e >> 1)] = acc[e] * factor[r];
    }
  }
  __syncthreads();
  // a warp's row, four outputs a lane
  const int r = warp, i = 4 * lane;
  if (rows.id[r] == kOutside || i >= cols || (rows.id[r] == kNone && p.base == p.out)) return;
  float4 v = rows.id[r] >= 0 ? *reinterpret_cast<const float4*>(&tile[r][i]) : make_float4(0.f, 0.f, 0.f, 0.f);
  const long long at = left + col + i;
  O* out = static_cast<O*>(p.out) + p.out_stride * (row0 + r) + at;
  const O* base = p.base ? static_cast<const O*>(p.base) + p.base_stride * (row0 + r) + at : nullptr;
  if constexpr (std::is_same<O, float>::value) {
    if (base) {
      const float4 b = *reinterpret_cast<const float4*>(base);
      if (rows.id[r] < 0) v = b;   // (base's own bits)
      else { v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w; }
    }
    *reinterpret_cast<float4*>(out) = v;
  } else {
    __align__(8) O w[4] = {to<O>(0.f), to<O>(0.f), to<O>(0.f), to<O>(0.f)};
    if (base) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(base);
    if (rows.id[r] >= 0) {
      w[0] = to<O>(from(w[0]) + v.x);
      w[1] = to<O>(from(w[1]) + v.y);
      w[2] = to<O>(from(w[2]) + v.z);
      w[3] = to<O>(from(w[3]) + v.w);
    }
    *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(w);
  }
}

template <class T>
cudaError_t launch(const AdaptParams& p, cudaStream_t st) {
  const int blocks = (p.rows + R - 1) / R;
  cudaError_t e = launch_k(shrink_kernel<T>, dim3(blocks, p.ksplit), kThreads, 0, st, p);
  if (e != cudaSuccess) return e;
  int tiles = 0;
  for (int j = 0; j < p.site.n_parts; ++j) tiles += (p.site.cols[j] + kTileCols - 1) / kTileCols;
  const dim3 grid(blocks, tiles);
  if (p.out_type != KVR_ACT_F32) return launch_k(expand_kernel<T, T, 2>, grid, kThreads, 0, st, p);
  constexpr int kTerms = std::is_same<T, __half>::value ? 2 : 3;
  return launch_k(expand_kernel<T, float, kTerms>, grid, kThreads, 0, st, p);
}

int adapt_split(const kvr_adapter_site& s, int rows, int sms) {
  const int blocks = (rows + R - 1) / R;
  const int most = std::max(1, std::min(kAdaptMaxSplit, s.k / 128));
  return std::max(1, std::min(most, 2 * sms / blocks));
}

}  // namespace

size_t adapt_work_bytes(const kvr_adapter_site& s, int rows) {
  // (of any number of SMs)
  return (size_t)adapt_split(s, rows, 1024) * rows * s.n_parts * s.max_rank * sizeof(float);
}

cudaError_t launch_adapt(AdaptParams p, int sms, cudaStream_t st) {
  p.ksplit = adapt_split(p.site, p.rows, std::min(sms, 1024));
  return p.site.type == KVR_ACT_F16 ? launch<__half>(p, st) : launch<__nv_bfloat16>(p, st);
}

}  // namespace kvr
