// Internal declarations of the paged 4-bit cache (include/kvr.h).
#pragma once

#include "kvr_internal.cuh"

namespace kvr {

constexpr int kPage = KVR_PAGE_TOKENS;   // tokens of a page
constexpr int kPageGroup = 32;           // elements along the head dimension that share a scale
constexpr float kPageScaleMax = 8188.f;  // 8 * 8188 = 65504: every value c * s has an fp16 number's magnitude
constexpr int kPageMaxSeqs = 2048;
// A score in log2 units that is larger makes its row NaN, one below minus it weighs nothing: 32
// bits place such numbers 32 apart and more, which leaves no weights.
constexpr float kScoreMax = 268435456.f;   // 2^28

// One page of one KV head ("chunk"), in the order the tensor-core fragments
// want it.  Key = token within the page, g = 0..7 and t = 0..3 the lane
// coordinates of an m16n8k16 fragment, j the groups of 32 dims.
//   K codes  [key][t][j] 32-bit words: dims 32 j + 8 t + 0..7 of the key.  Dims
//            2r and 2r + 1 of the eight sit in nibbles r and r + 4, so one bit
//            mask on a word gives two neighbouring dims as a 16-bit pair.
//   V codes  [key / 8][g][t][j] words: keys 8 (key / 8) + 2t (low half) and
//            2t + 1 (high half), nibble n of a half is dim 32 j + 4 g + n.
//            (Every 16-bit unit belongs to one token: an append never shares a
//            store with another token.)
//   K scales [key][j] fp16.
//   V scales [key / 16][t][(key / 8) % 2][j] pairs of fp16 (keys 2t, 2t + 1).
// A code is held with 8 added.  K codes and scales come first, so that K and V
// can be fetched apart, each as one run of kHalf bytes.
template <int D>
struct Chunk {
  static constexpr int kGroups = D / kPageGroup;
  static constexpr int kCodes = kPage * D / 2;
  static constexpr int kScales = kPage * kGroups * 2;
  static constexpr int kKs = kCodes;
  static constexpr int kHalf = kCodes + kScales;
  static constexpr int kV = kHalf;
  static constexpr int kVs = kHalf + kCodes;
  static constexpr int kBytes = 2 * kHalf;

  static __host__ __device__ __forceinline__ int k_word(int key, int t, int j) {
    return ((key * 4 + t) * kGroups + j) * 4;
  }
  static __host__ __device__ __forceinline__ int v_unit(int key, int g, int j) {
    return kV + ((((key >> 3) * 8 + g) * 4 + ((key >> 1) & 3)) * kGroups + j) * 4 + (key & 1) * 2;
  }
  static __host__ __device__ __forceinline__ int k_scale(int key, int j) { return kKs + (key * kGroups + j) * 2; }
  static __host__ __device__ __forceinline__ int v_scale(int key, int j) {
    return kVs + ((((key >> 4) * 4 + ((key >> 1) & 3)) * 2 + ((key >> 3) & 1)) * kGroups + j) * 4 + (key & 1) * 2;
  }
};

// the handle's configuration, device and planned rows (kvr_pages.cu)
const kvr_pages_config& pages_config(const kvr_pages* pages);
int pages_device(const kvr_pages* pages);
int pages_rows(const kvr_pages* pages);

inline size_t page_chunk_bytes(int d) { return d == 128 ? Chunk<128>::kBytes : Chunk<64>::kBytes; }

// What every kernel of the paged cache gets (device pointers of the work area).
struct PagesDev {
  uint8_t* pool;
  long long layer_off;   // bytes before this layer
  int32_t* table;        // [max_seqs][width]
  int32_t* lens;
  int32_t* free_list;
  int32_t* count;
  int32_t* cu;           // [max_seqs + 1]
  int32_t* row_seq;
  int32_t* row_pos;
  int32_t* row_slot;
  int32_t* info;         // [2]: sequences and rows of the last plan
  const float2* rope;    // [max_len][d / 2] (cos, sin)
  const __half2* rope_rest;   // what those rounded off, times 2^24
  int* status;           // a wait that gave up
  int* refused;          // the first refused plan's error code
  int n_pages, width, max_len, max_rows, max_seqs;
  int Hq, Hkv, G, d;
  uint32_t mul_hkv, mul_g;   // for dev::div_by
  int f16;               // activations are fp16 (else bf16)
};

struct PageAppend {
  const void* q;
  const void* k;
  const void* v;
  long long qs, ks, vs;      // row strides in elements
  const void* norm_q;
  const void* norm_k;
  void* q_out;
  int rotate, rows;
  float eps;
  int ctas_q, ctas_kv;       // CTAs of a row group for the heads of q, and of k and v each
};

// A segment of the tensor-memory kernel (a sequence, pair of row tiles and KV
// head) that several of its CTAs share: the first of them describes it.
struct PageShared {
  int parts;               // CTAs that share it, from this one on; 0: none
  int row0, R, tile, kv;   // first row and G * rows of the sequence
  int pad[3];
};

// Attention of the sequences with G * rows <= many (the split kernel).  The
// same launch merges what the tensor-memory kernel left in parts before it.
struct PageAttend {
  const void* q;
  long long qs;
  void* out;
  int out_f16;
  int rows;
  int many;
  float scale_log2;
  float* part;       // partial outputs
  float2* ml;        // their (the exponent that the weights are taken under, sum)
  int* counters;     // arrivals, zero between launches
  const PageShared* shared;   // [CTAs] of the tensor-memory kernel, null where it did not run
  const float* tc_part;
  const float2* tc_ml;
};

// ... and of the sequences with more (the tensor-memory kernel).
struct PageAttendTc {
  const void* q;
  long long qs;
  void* out;
  int out_f16;
  int rows;
  int many;
  int min_units;     // key blocks a CTA takes at least
  float scale_log2;
  // parts of segments: [CTAs][2][256 rows], first the one that began in an
  // earlier CTA, then the one that goes on in the next
  float* part;       // [d]
  float2* ml;        // (the exponent that the weights are taken under, their sum)
  PageShared* shared;
};
constexpr int kPageTcRows = 256;

constexpr int kPageAttnMaxCtas = 160;
constexpr int kPageTcPartRows = kPageAttnMaxCtas * 2 * kPageTcRows;
// partial results of the split kernel, in rows: two tiles of 8 for each of 16 warps
// and two per CTA
constexpr int kPageAttnPartRows = kPageAttnMaxCtas * (2 * 128 + 2 * 8);

cudaError_t page_plan_setup();
// every page free, the first ones on top
cudaError_t launch_page_init(const PagesDev& p, cudaStream_t st);
cudaError_t launch_page_rope(const RopeFreq& fr, int max_len, int d, float2* table, __half2* rest, cudaStream_t st);
cudaError_t launch_page_plan(const PagesDev& p, int n_seq, const int32_t* keep, const int32_t* add, int rows,
                             int max_add, cudaStream_t st);
cudaError_t launch_page_append(const PagesDev& p, PageAppend a, cudaStream_t st);
cudaError_t launch_page_read(const PagesDev& p, void* k_out, void* v_out, int rows, cudaStream_t st);
cudaError_t page_attn_setup();
cudaError_t launch_page_attn(const PagesDev& p, const PageAttend& a, int ctas, cudaStream_t st);
cudaError_t page_attn_tc_setup();
cudaError_t launch_page_attn_tc(const PagesDev& p, const PageAttendTc& a, int ctas, cudaStream_t st);

}  // namespace kvr

#ifdef __CUDACC__
namespace kvr {
namespace dev {

// n / d for n < 2^32 / d, with mul = ceil(2^32 / d) (0 stands for d = 1)
__device__ __forceinline__ int div_by(int n, uint32_t mul) { return mul ? (int)__umulhi((uint32_t)n, mul) : n; }

// two fp32 lanes in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}

__device__ __forceinline__ float2 neg2(float2 a) { return mul2(a, make_float2(-1.f, -1.f)); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.f, -1.f), a); }

// two activations of either 16-bit type
template <bool F16>
__device__ __forceinline__ float2 act2(uint32_t u) {
  if (F16) return __half22float2(*reinterpret_cast<__half2*>(&u));
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack_act(float lo, float hi) {
  if (F16) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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
// a number or, for NaN, 0 (scales are not negative)
__device__ __forceinline__ uint32_t number2(uint32_t s) {
  __half2 r = __hmax2(*reinterpret_cast<__half2*>(&s), __float2half2_rn(0.f));
  return *reinterpret_cast<uint32_t*>(&r);
}
// a register with a constant that the compiler does not form anew at each use
__device__ __forceinline__ uint32_t held(uint32_t x) {
  asm volatile("" : "+r"(x));
  return x;
}

}  // namespace dev
}  // namespace kvr
#endif
