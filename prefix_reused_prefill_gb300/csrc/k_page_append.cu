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
__device__ __forceinline__ void unpack8(uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = dev::act2<F16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(dev::pack_act<F16>(x[0], x[1]), dev::pack_act<F16>(x[2], x[3]),
                    dev::pack_act<F16>(x[4], x[5]), dev::pack_act<F16>(x[6], x[7]));
}

// codes (with 8 added) of 8 of the 32 elements of a group held by 4
// neighbouring lanes, and the group's scale.  The division is the exact one:
// a quotient halfway between two codes is common (16-bit values over a 16-bit
// scale) and goes to the even one.
__device__ __forceinline__ __half quantise8(const float* x, uint32_t* code) {
  // |x| as bits, so that NaN ranks above infinity and infinity above numbers
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (top >= 0x7f800000u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) code[i] = 8;
    return __ushort_as_half((unsigned short)0x7fffu);
  }
  const __half s = __float2half_rn(fminf(__fdiv_rn(__uint_as_float(top), 7.f), kPageScaleMax));
  const float sf = __half2float(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = sf > 0.f ? rintf(__fdiv_rn(x[i], sf)) : 0.f;
    code[i] = (uint32_t)((int)fminf(fmaxf(c, -8.f), 7.f) + 8);
  }
  return s;
}

template <int D, bool F16>
__global__ void __launch_bounds__(32 * kWarps)
page_append_kernel(const PagesDev p, const PageAppend a) {
  using C = Chunk<D>;
  using L = Lanes<D>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % L::kPer, t = l & 3;
  const int row = (int)blockIdx.x * L::kRows + lane / L::kPer;
  dev::pdl_trigger();
  dev::pdl_wait();
  const int total = min(a.rows, p.info[1]);
  if ((int)blockIdx.x * L::kRows >= total) return;
  const bool live = row < total;
  const int pos = live ? p.row_pos[row] : 0;
  const int slot = live ? p.row_slot[row] : 0;
  float2 cs[8];
  if (a.rotate) {
    const float4* src = reinterpret_cast<const float4*>(p.rope + (long long)pos * (D / 2) + 8 * l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = src[i];
      cs[2 * i] = make_float2(v.x, v.y);
      cs[2 * i + 1] = make_float2(v.z, v.w);
    }
  }
  const int h0 = a.q ? 0 : p.Hq;
  const int heads = p.Hq + 2 * p.Hkv;
  uint8_t* page = p.pool + p.layer_off + (long long)(slot / kPage) * p.Hkv * C::kBytes;
  const int key = slot % kPage;
  for (int h = h0 + (int)blockIdx.y * kWarps + warp; h < heads; h += kWarps * (int)gridDim.y) {
    const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
    const int hh = is_q ? h : (is_k ? h - p.Hq : h - p.Hq - p.Hkv);
    const uint16_t* src = static_cast<const uint16_t*>(is_q ? a.q : (is_k ? a.k : a.v));
    const long long stride = is_q ? a.qs : (is_k ? a.ks : a.vs);
    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
    if (live) {
      src += (long long)row * stride + hh * D + 8 * l;
      u0 = *reinterpret_cast<const uint4*>(src);
      u1 = *reinterpret_cast<const uint4*>(src + D / 2);
    }
    float x[16];
    unpack8<F16>(u0, x);
    unpack8<F16>(u1, x + 8);
    if (is_q || is_k) {
      const void* gain = is_q ? a.norm_q : a.norm_k;
      if (gain) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int m = 1; m < L::kPer; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float r = __fdiv_rn(1.f, __fsqrt_rn(ss * (1.f / D) + a.eps));
        const uint16_t* gp = static_cast<const uint16_t*>(gain) + 8 * l;
        float g[16];
        unpack8<F16>(*reinterpret_cast<const uint4*>(gp), g);
        unpack8<F16>(*reinterpret_cast<const uint4*>(gp + D / 2), g + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * r * g[i];
      }
      if (a.rotate) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float lo = x[i], hi = x[8 + i];
          x[i] = lo * cs[i].x - hi * cs[i].y;
          x[8 + i] = hi * cs[i].x + lo * cs[i].y;
        }
      }
      u0 = pack8<F16>(x);
      u1 = pack8<F16>(x + 8);
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
      unpack8<F16>(u1, x + 8);
    }
    uint8_t* chunk = page + (long long)hh * C::kBytes;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int j = part * (C::kGroups / 2) + l / 4;
      uint32_t c[8];
      const __half s = quantise8(x + 8 * part, c);
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
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
      float x[8];
      if (is_k) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(chunk + C::k_word(key, t, j));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[2 * r] = (float)((int)((w >> (4 * r)) & 15u) - 8) * s;
          x[2 * r + 1] = (float)((int)((w >> (4 * r + 16)) & 15u) - 8) * s;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w = *reinterpret_cast<const uint16_t*>(chunk + C::v_unit(key, 2 * t + e, j));
#pragma unroll
          for (int n = 0; n < 4; ++n) x[4 * e + n] = (float)((int)((w >> (4 * n)) & 15u) - 8) * s;
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
