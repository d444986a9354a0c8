// The planned rows of one layer (kvr_page_append): per head
//   y = x / sqrt(mean x^2 + eps) * gain      (q and k, where a gain is given)
//   (y_j, y_(j + d/2)) -> (y_j c - y_(j+d/2) s, y_(j+d/2) c + y_j s)
// in 32 bits, rounded once to the activation type, q written out, k and v
// quantised into their page: one read of the projection's output and one write.
//
// Bound by HBM bytes.  d / 16 lanes hold a head's vector, lane l the elements
// 8 l .. 8 l + 7 of both halves: 16-byte loads and stores, the rotation pairs in
// one lane, a group of 32 in four neighbouring lanes, a K code word in one
// lane.  A warp takes 32 / (d / 16) consecutive rows of the same head, which in
// a prompt are neighbouring tokens of a page, so that the 2-byte units of V
// (a unit never holds two tokens) meet in one 32-byte sector; it keeps the
// rows' cosines and sines in registers over the heads it walks.
//
// 8.2k rows of 32 + 2 * 8 heads of 128 with norms: 42 us, 4.2 TB/s of 176 MB, 62 % of
// a plain copy's rate; the quantising costs 3 us of it.  One to 254 rows: 3 to
// 4 us, a launch.
#include "kvr_pages.cuh"

namespace kvr {

namespace {

constexpr int kWarps = 8;

template <int D>
struct Lanes {
  static constexpr int kPer = D / 16;        // lanes of a vector
  static constexpr int kRows = 32 / kPer;    // rows of a warp
};

template <bool F16>
__device__ __forceinline__ void unpack8(uint4 u, float2* x) {
  x[0] = dev::act2<F16>(u.x);
  x[1] = dev::act2<F16>(u.y);
  x[2] = dev::act2<F16>(u.z);
  x[3] = dev::act2<F16>(u.w);
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float2* x) {
  return make_uint4(dev::pack_act<F16>(x[0].x, x[0].y), dev::pack_act<F16>(x[1].x, x[1].y),
                    dev::pack_act<F16>(x[2].x, x[2].y), dev::pack_act<F16>(x[3].x, x[3].y));
}

// 1.5 * 2^23: adding it rounds a small number to an integer, halves to the even
// one, and leaves that integer in the low bits
constexpr float kRound = 12582912.f;

// code (with 8 added) of x under the scale s: x / s rounded, halves to the even
// code, at most [-8, 7].  x times 1 / s can be off by 2^-23 of itself, and a
// quotient exactly halfway is common (16-bit values over a 16-bit scale): the
// remainder x - n s, which an FMA gives exactly, tells where n is to be moved.
__device__ __forceinline__ uint32_t code_of(float x, float s, float inv, float half) {
  float t = fminf(fmaxf(x * inv, -9.f), 9.f) + kRound;
  const float d = fmaf(kRound - t, s, x);
  if (fabsf(d) >= half && (fabsf(d) > half || (__float_as_uint(t) & 1u))) t += d > 0.f ? 1.f : -1.f;
  t = fminf(fmaxf(t, kRound - 8.f), kRound + 7.f);
  return __float_as_uint(t) - (__float_as_uint(kRound) - 8u);
}

// codes of 8 of the 32 elements of a group held by 4 neighbouring lanes, and the
// group's scale
__device__ __forceinline__ __half quantise8(const float2* x, uint32_t* code) {
  // |x| as bits, so that NaN ranks above infinity and infinity above numbers
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    top = max(top, max(__float_as_uint(x[i].x) & 0x7fffffffu, __float_as_uint(x[i].y) & 0x7fffffffu));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const bool bad = top >= 0x7f800000u;
  const __half s = __float2half_rn(bad ? 0.f : fminf(__fdiv_rn(__uint_as_float(top), 7.f), kPageScaleMax));
  const float sf = __half2float(s);
  // (without a scale every code is 0: no remainder passes an infinite half)
  const float inv = sf > 0.f ? __frcp_rn(sf) : 0.f, half = sf > 0.f ? 0.5f * sf : INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    code[2 * i] = code_of(bad ? 0.f : x[i].x, sf, inv, half);
    code[2 * i + 1] = code_of(bad ? 0.f : x[i].y, sf, inv, half);
  }
  return bad ? __ushort_as_half((unsigned short)0x7fffu) : s;
}

template <int D, bool F16>
__global__ void __launch_bounds__(32 * kWarps, 4)
page_append_kernel(const PagesDev p, const PageAppend a) {
  using C = Chunk<D>;
  using L = Lanes<D>;
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int l = lane % L::kPer, t = l & 3;
  const int row = (int)blockIdx.x * L::kRows + lane / L::kPer;
  dev::pdl_trigger();
  dev::pdl_wait();
  const int total = min(a.rows, p.info[1]);
  if ((int)blockIdx.x * L::kRows >= total) return;
  const bool live = row < total;
  const int pos = live ? p.row_pos[row] : 0;
  const int slot = live ? p.row_slot[row] : 0;
  float2 cs[4], sn[4];   // cosines and sines of dims 8 l .. 8 l + 7
  if (a.rotate) {
    const float4* src = reinterpret_cast<const float4*>(p.rope + (long long)pos * (D / 2) + 8 * l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = src[i];
      cs[i] = make_float2(v.x, v.z);
      sn[i] = make_float2(v.y, v.w);
    }
  }
  const int h0 = a.q ? 0 : p.Hq;
  const int heads = p.Hq + 2 * p.Hkv;
  uint8_t* page = p.pool + p.layer_off + (long long)(slot / kPage) * p.Hkv * C::kBytes;
  const int key = slot % kPage;
  // this lane's elements of head h of its row.  The next head's are asked for
  // before this one's are used (in the example of the head 61 us without, 51 us
  // so, 44 us with the exact division replaced and four CTAs on an SM; without
  // any quantising 41 us)
  auto fetch = [&](int h, uint4& lo, uint4& hi) {
    if (!live || h >= heads) return;
    const uint16_t* src;
    if (h < p.Hq) src = static_cast<const uint16_t*>(a.q) + (long long)row * a.qs + h * D;
    else if (h < p.Hq + p.Hkv) src = static_cast<const uint16_t*>(a.k) + (long long)row * a.ks + (h - p.Hq) * D;
    else src = static_cast<const uint16_t*>(a.v) + (long long)row * a.vs + (h - p.Hq - p.Hkv) * D;
    lo = __ldcs(reinterpret_cast<const uint4*>(src + 8 * l));
    hi = __ldcs(reinterpret_cast<const uint4*>(src + 8 * l + D / 2));
  };
  const int step = kWarps * (int)gridDim.y;
  int h = h0 + (int)blockIdx.y * kWarps + warp;
  uint4 next0 = make_uint4(0, 0, 0, 0), next1 = next0;
  fetch(h, next0, next1);
  for (; h < heads; h += step) {
    const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
    const int hh = is_q ? h : (is_k ? h - p.Hq : h - p.Hq - p.Hkv);
    uint4 u0 = next0, u1 = next1;
    fetch(h + step, next0, next1);
    float2 x[8];
    unpack8<F16>(u0, x);
    unpack8<F16>(u1, x + 4);
    if (is_q || is_k) {
      const void* gain = is_q ? a.norm_q : a.norm_k;
      if (gain) {
        float2 s2 = dev::mul2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) s2 = dev::fma2(x[i], x[i], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int m = 1; m < L::kPer; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float r = rsqrtf(ss * (1.f / D) + a.eps);   // (2 ulp)
        const uint16_t* gp = static_cast<const uint16_t*>(gain) + 8 * l;
        float2 g[8];
        unpack8<F16>(*reinterpret_cast<const uint4*>(gp), g);
        unpack8<F16>(*reinterpret_cast<const uint4*>(gp + D / 2), g + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = dev::mul2(dev::mul2(x[i], make_float2(r, r)), g[i]);
      }
      if (a.rotate) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 lo = x[i], hi = x[4 + i];
          x[i] = dev::fma2(lo, cs[i], dev::mul2(hi, make_float2(-sn[i].x, -sn[i].y)));
          x[4 + i] = dev::fma2(hi, cs[i], dev::mul2(lo, sn[i]));
        }
      }
      u0 = pack8<F16>(x);
      u1 = pack8<F16>(x + 4);
      if (is_q) {
        if (live) {
          uint16_t* dst = static_cast<uint16_t*>(a.q_out) + ((long long)row * p.Hq + hh) * D + 8 * l;
          *reinterpret_cast<uint4*>(dst) = u0;
          *reinterpret_cast<uint4*>(dst + D / 2) = u1;
        }
        continue;
      }
      // the values that the cache quantises are those of the activation type
      unpack8<F16>(u0, x);
      unpack8<F16>(u1, x + 4);
    }
    uint8_t* chunk = page + (long long)hh * C::kBytes;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int j = part * (C::kGroups / 2) + l / 4;
      uint32_t c[8];
      const __half s = quantise8(x + 4 * part, c);
      if (!live) continue;
      if (is_k) {
        uint32_t w = 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) w |= (c[2 * r] << (4 * r)) | (c[2 * r + 1] << (4 * r + 16));
        *reinterpret_cast<uint32_t*>(chunk + C::k_word(key, t, j)) = w;
        if (t == 0) *reinterpret_cast<__half*>(chunk + C::k_scale(key, j)) = s;
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w = c[4 * e] | (c[4 * e + 1] << 4) | (c[4 * e + 2] << 8) | (c[4 * e + 3] << 12);
          *reinterpret_cast<uint16_t*>(chunk + C::v_unit(key, 2 * t + e, j)) = (uint16_t)w;
        }
        if (t == 0) *reinterpret_cast<__half*>(chunk + C::v_scale(key, j)) = s;
      }
    }
  }
}

// The values of the planned rows: the same lanes, the other way round.
template <int D, bool F16>
__global__ void __launch_bounds__(32 * kWarps)
page_read_kernel(const PagesDev p, void* k_out, void* v_out, int rows) {
  using C = Chunk<D>;
  using L = Lanes<D>;
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int l = lane % L::kPer, t = l & 3;
  const int row = (int)blockIdx.x * L::kRows + lane / L::kPer;
  dev::pdl_trigger();
  dev::pdl_wait();
  if (row >= min(rows, p.info[1])) return;
  const int slot = p.row_slot[row], key = slot % kPage;
  const uint8_t* page = p.pool + p.layer_off + (long long)(slot / kPage) * p.Hkv * C::kBytes;
  for (int h = (int)blockIdx.y * kWarps + warp; h < 2 * p.Hkv; h += kWarps * (int)gridDim.y) {
    const bool is_k = h < p.Hkv;
    const int hh = is_k ? h : h - p.Hkv;
    const uint8_t* chunk = page + (long long)hh * C::kBytes;
    uint16_t* dst = static_cast<uint16_t*>(is_k ? k_out : v_out) + ((long long)row * p.Hkv + hh) * D + 8 * l;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int j = part * (C::kGroups / 2) + l / 4;
      const float s =
          __half2float(*reinterpret_cast<const __half*>(chunk + (is_k ? C::k_scale(key, j) : C::v_scale(key, j))));
      float2 x[4];
      auto value = [&](uint32_t w, int bit) { return (float)((int)((w >> bit) & 15u) - 8) * s; };
      if (is_k) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(chunk + C::k_word(key, t, j));
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = make_float2(value(w, 4 * r), value(w, 4 * r + 16));
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w = *reinterpret_cast<const uint16_t*>(chunk + C::v_unit(key, 2 * t + e, j));
          x[2 * e] = make_float2(value(w, 0), value(w, 4));
          x[2 * e + 1] = make_float2(value(w, 8), value(w, 12));
        }
      }
      *reinterpret_cast<uint4*>(dst + part * (D / 2)) = pack8<F16>(x);
    }
  }
}

// CTAs: a row group each, its heads split over as many as fill the card
dim3 row_grid(int rows, int per, int heads) {
  const int groups = (rows + per - 1) / per;
  const int most = (heads + kWarps - 1) / kWarps;
  const int want = (1216 + groups - 1) / groups;
  return dim3(groups, most < want ? most : want);
}

}  // namespace

cudaError_t launch_page_append(const PagesDev& p, const PageAppend& a, cudaStream_t st) {
  const int heads = (a.q ? p.Hq : 0) + 2 * p.Hkv;
  const dim3 grid = row_grid(a.rows, p.d == 128 ? Lanes<128>::kRows : Lanes<64>::kRows, heads);
  if (p.d == 128)
    return p.f16 ? launch_k(page_append_kernel<128, true>, grid, 32 * kWarps, 0, st, p, a)
                 : launch_k(page_append_kernel<128, false>, grid, 32 * kWarps, 0, st, p, a);
  return p.f16 ? launch_k(page_append_kernel<64, true>, grid, 32 * kWarps, 0, st, p, a)
               : launch_k(page_append_kernel<64, false>, grid, 32 * kWarps, 0, st, p, a);
}

cudaError_t launch_page_read(const PagesDev& p, void* k_out, void* v_out, int rows, cudaStream_t st) {
  const dim3 grid = row_grid(rows, p.d == 128 ? Lanes<128>::kRows : Lanes<64>::kRows, 2 * p.Hkv);
  if (p.d == 128)
    return p.f16 ? launch_k(page_read_kernel<128, true>, grid, 32 * kWarps, 0, st, p, k_out, v_out, rows)
                 : launch_k(page_read_kernel<128, false>, grid, 32 * kWarps, 0, st, p, k_out, v_out, rows);
  return p.f16 ? launch_k(page_read_kernel<64, true>, grid, 32 * kWarps, 0, st, p, k_out, v_out, rows)
               : launch_k(page_read_kernel<64, false>, grid, 32 * kWarps, 0, st, p, k_out, v_out, rows);
}

}  // namespace kvr
