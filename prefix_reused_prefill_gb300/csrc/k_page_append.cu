// The planned rows of one layer (kvr_page_append): per head
//   y = x / sqrt(mean x^2 + eps) * gain      (q and k, where a gain is given)
//   (y_j, y_(j + d/2)) -> (y_j c - y_(j+d/2) s, y_(j+d/2) c + y_j s)
// rounded to the activation type, q written out, k and v quantised into their
// page: one read of the projection's output and one write.  q is formed in 32
// bits, k in sums of two floats: a rounding to the other side of a border may move a
// code, and that is 1 / 7 of the group's largest value.
//
// d / 16 lanes hold a head's vector, lane l the elements 8 l .. 8 l + 7 of both
// halves: 16-byte loads and stores, the rotation pairs in one lane, a group of
// 32 in four neighbouring lanes, a K code word in one lane.  A warp takes
// 32 / (d / 16) consecutive rows of the same head, which in a prompt are
// neighbouring tokens of a page, so that the 2-byte units of V (a unit never
// holds two tokens) meet in one 32-byte sector.
//
// 8.2k rows of 32 + 2 * 8 heads of 128 with norms: 42.9 us, 4.1 TB/s of 176 MB, 61 %
// of a plain copy's rate, with the issue slots 63 % busy and waits for loads the longest
// (3.0 warps of 6.5 an issue): each CTA has one row group and little after its start of
// dependent loads.  k's second floats take 6 us (with them k is that of 64 bits in all
// of 50 million values, in 32 bits two or three codes in 8 million moved); more loads
// in flight (through shared memory) or more CTAs for q change nothing.  q, k and v in one loop
// of the same CTAs: 47.8.  One to 254 rows: 3 to 4 us, a launch.
#include "kvr_pages.cuh"

namespace kvr {

namespace {

// 7 CTAs of 4 warps on an SM: 72 registers, which nothing is spilled from (each
// spilled word is a store past L1: 100 bytes of them a thread made it 66 us and more)
constexpr int kWarps = 4;

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

// minus the code of x under the scale s, whatever they are: x / s rounded, halves to
// the even number, at most [-8, 7].  A quotient exactly halfway goes to the even
// one by the remainder.
__device__ __forceinline__ float minus_code(float x, float s, float inv) {
  const float half = s > 0.f ? 0.5f * s : INFINITY;
  float t = fminf(fmaxf(x * inv, -9.f), 9.f) + kRound;
  const float d = fmaf(kRound - t, s, x);
  if (fabsf(d) >= half && (fabsf(d) > half || (__float_as_uint(t) & 1u))) t += d > 0.f ? 1.f : -1.f;
  return fminf(fmaxf(kRound - t, -7.f), 8.f);
}

// the larger of |a| and |b|, element by element; NaN where either is
template <bool F16>
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
  a &= 0x7fff7fffu;
  b &= 0x7fff7fffu;
  if (F16) {
    const __half2 m = __hmax2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Codes of 8 of the 32 elements of a group held by 4 neighbouring lanes (u: as they
// are, x: as floats), and the group's scale.  of_k: a word of K (elements 0, 2, 4,
// 6 in its lower half); else two units of V, 4 elements each, side by side.
template <bool F16>
__device__ __forceinline__ __half quantise8(uint4 u, const float2* x, bool of_k, uint32_t& word) {
  uint32_t m = abs_max2<F16>(abs_max2<F16>(u.x, u.y), abs_max2<F16>(u.z, u.w));
  m = abs_max2<F16>(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = abs_max2<F16>(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const float2 tops = dev::act2<F16>(m);
  const bool bad = !(tops.x < INFINITY && tops.y < INFINITY);
  const float top = fmaxf(tops.x, tops.y);
  const __half s = __float2half_rn(bad ? 0.f : fminf(__fdiv_rn(top, 7.f), kPageScaleMax));
  const float sf = __half2float(s);
  const float inv = sf > 0.f ? __frcp_rn(sf) : 0.f;   // (without a scale every code is 0)
  // -round(x / s), halves to the even number.  x times 1 / s can be off by 2^-23 of
  // itself, and a quotient exactly halfway is common (16-bit values over a 16-bit
  // scale; 4 groups of 100): the remainder x - n s, which an FMA gives exactly, is
  // either exactly half of s or 2^-12 s from it, so rounded to 2^-14 s it is added to n
  // without error.  A scale that is neither cut nor subnormal is top / 7 to 2^-11: no
  // code passes 7.
  constexpr float kFine = 768.f;   // 1.5 2^9: sums with it are multiples of 2^-14
  float2 n[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 whole = make_float2(kRound, kRound), fine = make_float2(kFine, kFine);
    const float2 t = dev::fma2(x[i], make_float2(inv, inv), whole);
    const float2 d = dev::fma2(dev::sub2(whole, t), make_float2(sf, sf), x[i]);
    const float2 e = dev::sub2(dev::fma2(d, make_float2(inv, inv), fine), fine);
    n[i] = dev::sub2(whole, dev::add2(t, e));
  }
  if (bad || sf == kPageScaleMax || (sf > 0.f && sf < 6.103515625e-5f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = i & 1 ? x[i / 2].y : x[i / 2].x;
      const float c = minus_code(bad ? 0.f : v, sf, inv);
      if (i & 1) n[i / 2].y = c;
      else n[i / 2].x = c;
    }
  }
  // the codes (with 8 added) as exact sums of powers of 16
  if (of_k) {
    float2 sum = make_float2(8388608.f + 0x8888, 8388608.f + 0x8888);
    sum = dev::sub2(sum, n[0]);
    sum = dev::fma2(n[1], make_float2(-16.f, -16.f), sum);
    sum = dev::fma2(n[2], make_float2(-256.f, -256.f), sum);
    sum = dev::fma2(n[3], make_float2(-4096.f, -4096.f), sum);
    word = __byte_perm(__float_as_uint(sum.x), __float_as_uint(sum.y), 0x5410);
  } else {
    uint32_t w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float2 sum = dev::fma2(n[2 * e], make_float2(-1.f, -16.f), make_float2(8388608.f + 0x8888, 0.f));
      sum = dev::fma2(n[2 * e + 1], make_float2(-256.f, -4096.f), sum);
      w[e] = __float_as_uint(sum.x + sum.y);
    }
    word = __byte_perm(w[0], w[1], 0x5410);
  }
  return bad ? __ushort_as_half((unsigned short)0x7fffu) : s;
}

// Numbers as sums hi + lo of two floats (2^-45 or so), for k next to the border of
// two activation values: k is rounded to that type and then to a code, and on the
// other side of both borders it would move by a whole scale, 1 / 7 of the
// group's largest.
// a + b = hi + lo, exactly (Knuth's sum of two numbers and its error)
__device__ __forceinline__ void two_sum(float2 a, float2 b, float2& hi, float2& lo) {
  hi = dev::add2(a, b);
  const float2 v = dev::sub2(hi, a);
  lo = dev::add2(dev::sub2(a, dev::sub2(hi, v)), dev::sub2(b, v));
}
__device__ __forceinline__ void two_sum(float a, float b, float& hi, float& lo) {
  hi = a + b;
  const float v = hi - a;
  lo = (a - (hi - v)) + (b - v);
}
// 1 / sqrt(mean x^2 + eps) over the d elements of a head, 16 of them here
template <int D>
__device__ __forceinline__ float2 exact_rsqrt(const float2* x, float eps) {
  float2 s = dev::mul2(x[0], x[0]), rest = make_float2(0.f, 0.f);   // (16-bit numbers: exact squares)
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    float2 lo;
    two_sum(s, dev::mul2(x[i], x[i]), s, lo);
    rest = dev::add2(rest, lo);
  }
  float hi, lo;
  two_sum(s.x, s.y, hi, lo);
  lo += rest.x + rest.y;
#pragma unroll
  for (int m = 1; m < Lanes<D>::kPer; m <<= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, hi, m), other_lo = __shfl_xor_sync(0xffffffffu, lo, m);
    float e;
    two_sum(hi, other, hi, e);
    lo += other_lo + e;
  }
  float e;
  two_sum(hi * (1.f / D), eps, hi, e);
  lo = fmaf(lo, 1.f / D, e);
  // one step of Newton's from the approximate root, the residual 1 - v r^2 formed
  // from the exact product v r
  if (hi == INFINITY) return make_float2(0.f, 0.f);   // (the sum passed the largest number)
  const float r = rsqrtf(hi), p = hi * r, pe = fmaf(hi, r, -p);
  const float off = fmaf(-fmaf(lo, r, pe), r, fmaf(-p, r, 1.f));
  return make_float2(r, 0.5f * r * off);
}
// (a c - b s) r with cosines c, sines s and r of two parts each; na = -a, nb = -b
__device__ __forceinline__ float2 exact_turn(float2 a, float2 na, float2 b, float2 nb, float2 c, float2 s, float2 c_lo,
                                             float2 s_lo, bool scaled, float2 r) {
  const float2 p = dev::mul2(a, c), q = dev::mul2(nb, s);
  float2 hi, lo;
  two_sum(p, q, hi, lo);
  lo = dev::sub2(lo, dev::add2(dev::fma2(na, c, p), dev::fma2(b, s, q)));   // (less what p and q are too large)
  lo = dev::fma2(a, c_lo, lo);
  lo = dev::fma2(nb, s_lo, lo);
  if (scaled) {
    const float2 rr = make_float2(r.x, r.x), y = dev::mul2(hi, rr);
    lo = dev::fma2(lo, rr, dev::mul2(hi, make_float2(r.y, r.y)));
    lo = dev::sub2(lo, dev::fma2(hi, make_float2(-r.x, -r.x), y));
    hi = y;
  }
  return dev::add2(hi, lo);
}

template <int D, bool F16>
__global__ void __launch_bounds__(32 * kWarps, 7)
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
  // cosines and sines of this lane's dims 8 l .. 8 l + 7
  const float4* turns = reinterpret_cast<const float4*>(p.rope + (long long)pos * (D / 2) + 8 * l);
  const uint4* turns_rest = reinterpret_cast<const uint4*>(p.rope_rest + (long long)pos * (D / 2) + 8 * l);
  uint8_t* page = p.pool + p.layer_off + (long long)(slot / kPage) * p.Hkv * C::kBytes;
  const int key = slot % kPage;
  // body(head, this lane's elements of it) for this warp's share of n heads, those of
  // the CTAs y of ny.  The next head's are asked for before this one's are used
  // (61 -> 51 us in the example of the head).
  auto for_heads = [&](const void* base, long long stride, int n, int y, int ny, auto body) {
    const uint16_t* src = static_cast<const uint16_t*>(base) + (long long)row * stride + 8 * l;
    uint4 next0 = make_uint4(0, 0, 0, 0), next1 = next0;
    auto fetch = [&](int h) {
      if (!live || h >= n) return;
      next0 = __ldcs(reinterpret_cast<const uint4*>(src + h * D));
      next1 = __ldcs(reinterpret_cast<const uint4*>(src + h * D + D / 2));
    };
    int h = y * kWarps + warp;
    fetch(h);
    for (; h < n; h += kWarps * ny) {
      const uint4 u0 = next0, u1 = next1;
      fetch(h + kWarps * ny);
      body(h, u0, u1);
    }
  };
  // q, k and v in CTAs of their own: each then has the registers that it needs
  const int y = (int)blockIdx.y;
  if (y < a.ctas_q) {
    float2 cs[4], sn[4];
    if (a.rotate) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = turns[i];
        cs[i] = make_float2(v.x, v.z);
        sn[i] = make_float2(v.y, v.w);
      }
    }
    for_heads(a.q, a.qs, p.Hq, y, a.ctas_q, [&](int h, uint4 u0, uint4 u1) {
      float2 x[8];
      unpack8<F16>(u0, x);
      unpack8<F16>(u1, x + 4);
      if (a.norm_q) {
        float2 s2 = dev::mul2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) s2 = dev::fma2(x[i], x[i], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int m = 1; m < L::kPer; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float r = rsqrtf(ss * (1.f / D) + a.eps);   // (2 ulp)
        const uint16_t* gp = static_cast<const uint16_t*>(a.norm_q) + 8 * l;
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
      if (live) {
        uint16_t* dst = static_cast<uint16_t*>(a.q_out) + ((long long)row * p.Hq + h) * D + 8 * l;
        *reinterpret_cast<uint4*>(dst) = pack8<F16>(x);
        *reinterpret_cast<uint4*>(dst + D / 2) = pack8<F16>(x + 4);
      }
    });
  } else if (y < a.ctas_q + a.ctas_kv) {
    for_heads(a.k, a.ks, p.Hkv, y - a.ctas_q, a.ctas_kv, [&](int h, uint4 u0, uint4 u1) {
      float2 x[8];
      unpack8<F16>(u0, x);
      unpack8<F16>(u1, x + 4);
      if (a.norm_k || a.rotate) {
        float2 root = make_float2(1.f, 0.f);
        if (a.norm_k) {
          root = exact_rsqrt<D>(x, a.eps);
          const uint16_t* gp = static_cast<const uint16_t*>(a.norm_k) + 8 * l;
          const uint4 g[2] = {*reinterpret_cast<const uint4*>(gp), *reinterpret_cast<const uint4*>(gp + D / 2)};
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = dev::mul2(x[i], dev::act2<F16>(reinterpret_cast<const uint32_t*>(g)[i]));
        }
        if (a.rotate) {
          const uint4 w[2] = {turns_rest[0], turns_rest[1]};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 v = turns[i];
            const float2 e = dev::act2<true>(reinterpret_cast<const uint32_t*>(w)[2 * i]);
            const float2 f = dev::act2<true>(reinterpret_cast<const uint32_t*>(w)[2 * i + 1]);
            const float2 unit = make_float2(5.9604644775390625e-8f, 5.9604644775390625e-8f);   // 2^-24
            const float2 c_lo = dev::mul2(make_float2(e.x, f.x), unit), s_lo = dev::mul2(make_float2(e.y, f.y), unit);
            const float2 c = make_float2(v.x, v.z), s = make_float2(v.y, v.w), lo = x[i], hi = x[4 + i];
            const float2 nlo = dev::neg2(lo), nhi = dev::neg2(hi);
            x[i] = exact_turn(lo, nlo, hi, nhi, c, s, c_lo, s_lo, a.norm_k, root);
            x[4 + i] = exact_turn(hi, nhi, nlo, lo, c, s, c_lo, s_lo, a.norm_k, root);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 rr = make_float2(root.x, root.x), z = dev::mul2(x[i], rr);
            x[i] = dev::add2(z, dev::fma2(x[i], make_float2(root.y, root.y), dev::fma2(x[i], rr, dev::neg2(z))));
          }
        }
        u0 = pack8<F16>(x);
        u1 = pack8<F16>(x + 4);
        // the values that the cache quantises are those of the activation type
        unpack8<F16>(u0, x);
        unpack8<F16>(u1, x + 4);
      }
      uint8_t* chunk = page + (long long)h * C::kBytes;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const int j = part * (C::kGroups / 2) + l / 4;
        uint32_t word;
        const __half s = quantise8<F16>(part ? u1 : u0, x + 4 * part, true, word);
        if (!live) continue;
        *reinterpret_cast<uint32_t*>(chunk + C::k_word(key, t, j)) = word;
        if (t == 0) *reinterpret_cast<__half*>(chunk + C::k_scale(key, j)) = s;
      }
    });
  } else {
    for_heads(a.v, a.vs, p.Hkv, y - a.ctas_q - a.ctas_kv, a.ctas_kv, [&](int h, uint4 u0, uint4 u1) {
      float2 x[8];
      unpack8<F16>(u0, x);
      unpack8<F16>(u1, x + 4);
      uint8_t* chunk = page + (long long)h * C::kBytes;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const int j = part * (C::kGroups / 2) + l / 4;
        uint32_t word;
        const __half s = quantise8<F16>(part ? u1 : u0, x + 4 * part, false, word);
        if (!live) continue;
        *reinterpret_cast<uint16_t*>(chunk + C::v_unit(key, 2 * t, j)) = (uint16_t)word;
        *reinterpret_cast<uint16_t*>(chunk + C::v_unit(key, 2 * t + 1, j)) = (uint16_t)(word >> 16);
        if (t == 0) *reinterpret_cast<__half*>(chunk + C::v_scale(key, j)) = s;
      }
    });
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

cudaError_t launch_page_append(const PagesDev& p, PageAppend a, cudaStream_t st) {
  const int per = p.d == 128 ? Lanes<128>::kRows : Lanes<64>::kRows;
  dim3 grid = row_grid(a.rows, per, p.Hkv);
  a.ctas_kv = (int)grid.y;
  a.ctas_q = a.q ? (int)row_grid(a.rows, per, p.Hq).y : 0;
  grid.y = (unsigned)(a.ctas_q + 2 * a.ctas_kv);
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
