// weight.cuh - fixed-point softmax weights: exp((l - m) / T) as integers, so that sums of them are
// exact whatever their order, and the running mass that decides a drawn token does not depend on
// the grid, the cluster size or the order of atomics.
//
// w = 2^s with s = (l - m) * log2(e) / T <= 0, as an integer multiple of 2^-43 (at most 2^43, so
// 2^20 of them sum below 2^63). A drawn token changes where u * total falls within the error of the
// running mass of a border between two tokens. With fp32 exponentials (2^-22 relative) over 163840
// columns that is a row in a few dozen; here s is carried in two floats and 2^s to about 2^-39
// relative, which makes it one in millions, for about 50 instructions an element. FP64 would do
// too, but its rate here is 1/64 of FP32's.
//
// 2^s = 2^e * 2^(j/128) * 2^g with 128 s = 128 e + j + 128 g, |g| <= 2^-8: the table holds
// round(2^(j/128) * 2^43); 2^g - 1 is its Taylor series to the 4th order (the 5th is below 2^-49),
// its linear term in two floats. Weights below 2^-44 of the largest count as zero.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace tfd {

constexpr float kCutLog2 = -44.0f;         // below this s a weight is zero
constexpr int64_t kMaxDrawCols = 1 << 20;  // sums of this many weights stay at or below 2^63

__device__ const unsigned long long kExp2Table[128] = {
    0x80000000000ull, 0x80b1ed4fd9aull, 0x8164d1f3bc0ull, 0x8218af43740ull, 0x82cd8698ac3ull, 0x8383594eefbull,
    0x843a28c3aceull, 0x84f1f65637aull, 0x85aac367cc5ull, 0x8664915b924ull, 0x871f61969e9ull, 0x87db357ff6aull,
    0x88980e8092eull, 0x8955ee03619ull, 0x8a14d575497ull, 0x8ad4c6452c7ull, 0x8b95c1e3ea9ull, 0x8c57c9c4647ull,
    0x8d1adf5b7e6ull, 0x8ddf042022eull, 0x8ea4398b45dull, 0x8f6a8117e6dull, 0x9031dc43146ull, 0x90fa4c8beeeull,
    0x91c3d373ab1ull, 0x928e727d953ull, 0x935a2b2f13eull, 0x9426ff0fab2ull, 0x94f4efa8fefull, 0x95c3fe86d6dull,
    0x96942d37202ull, 0x97657d49f18ull, 0x9837f0518dcull, 0x990b87e266cull, 0x99e0459320bull, 0x9ab62afc950ull,
    0x9b8d39b9d55ull, 0x9c6573682ecull, 0x9d3ed9a72d0ull, 0x9e196e189d4ull, 0x9ef5326091aull, 0x9fd22825640ull,
    0xa0b0510fb97ull, 0xa18faeca854ull, 0xa27043030c5ull, 0xa3520f68e80ull, 0xa43515ae09eull, 0xa5195786beaull,
    0xa5fed6a9b15ull, 0xa6e594cfeefull, 0xa7cd93b4e96ull, 0xa8b6d5167b3ull, 0xa9a15ab4ea8ull, 0xaa8d2652ec9ull,
    0xab7a39b5a94ull, 0xac6896a4be4ull, 0xad583eea42aull, 0xae493452ca3ull, 0xaf3b78ad691ull, 0xb02f0dcbb6eull,
    0xb123f581d2bull, 0xb21a31a6662ull, 0xb311c412a91ull, 0xb40aaea2655ull, 0xb504f333f9eull, 0xb60093a85edull,
    0xb6fd91e328dull, 0xb7fbefca8caull, 0xb8fbaf47630ull, 0xb9fcd2452c1ull, 0xbaff5ab2134ull, 0xbc034a7ef2full,
    0xbd08a39f581ull, 0xbe0f6809861ull, 0xbf1799b67a7ull, 0xc0213aa1f0dull, 0xc12c4cca667ull, 0xc238d2311e4ull,
    0xc346ccda249ull, 0xc4563ecc533ull, 0xc5672a11550ull, 0xc67990b5aa2ull, 0xc78d74c8abcull, 0xc8a2d85c900ull,
    0xc9b9bd866e3ull, 0xcad2265e429ull, 0xcbec14fef27ull, 0xcd078b86504ull, 0xce248c151f8ull, 0xcf4318cf192ull,
    0xd06333daef3ull, 0xd184df62517ull, 0xd2a81d91f13ull, 0xd3ccf09985aull, 0xd4f35aabcffull, 0xd61b5dfe9faull,
    0xd744fccad6aull, 0xd870394c6dbull, 0xd99d15c278bull, 0xdacb946f2adull, 0xdbfbb797dafull, 0xdd2d8185083ull,
    0xde60f4825e1ull, 0xdf9612deb8full, 0xe0ccdeec2a9ull, 0xe2055afffe8ull, 0xe33f8972be9ull, 0xe47b6ca0374ull,
    0xe5b906e77c8ull, 0xe6f85aaaee2ull, 0xe8396a503c5ull, 0xe97c38406c5ull, 0xeac0c6e7dd2ull, 0xec0718b64c2ull,
    0xed4f301ed99ull, 0xee990f980daull, 0xefe4b99bdceull, 0xf13230a7ad1ull, 0xf281773c5a0ull, 0xf3d28fde3a6ull,
    0xf5257d15248ull, 0xf67a416c734ull, 0xf7d0df730adull, 0xf92959bb5ddull, 0xfa83b2db723ull, 0xfbdfed6ce5full,
    0xfd3e0c0cf48ull, 0xfe9e115c7b9ull,
};

// log2(e) / T in two floats; T below 1e-30 counts as 1e-30 (the quotient has to be a float).
struct Scale {
  float hi, lo;
};
__device__ __forceinline__ Scale scale_of(float t) {
  const float lh = 1.44269502e+00f, ll = 1.92596299e-08f;  // log2(e) = lh + ll to 2^-50
  t = fmaxf(t, 1e-30f);
  Scale c;
  c.hi = __fdiv_rn(lh, t);
  c.lo = __fdiv_rn(__fmaf_rn(-c.hi, t, lh) + ll, t);
  return c;
}

// The leading part of s, monotone in l (one subtraction, one product, both rounded): what bins and
// the zero cut go by.
__device__ __forceinline__ float lead_log2(float l, float m, const Scale& c) {
  return __fmul_rn(__fsub_rn(l, m), c.hi);
}
// Whether a column has a weight at all: NaN and what lies below the cut have none.
__device__ __forceinline__ bool alive(float ph) { return ph >= kCutLog2; }

// s = ph + pl: l - m in two floats (exact) times c in two floats. Finite for an alive column.
__device__ __forceinline__ float tail_log2(float l, float m, const Scale& c, float ph) {
  const float dh = __fsub_rn(l, m);
  const float bb = __fsub_rn(dh, l);
  const float dl = __fsub_rn(__fsub_rn(l, __fsub_rn(dh, bb)), __fadd_rn(m, bb));
  float pl = __fmaf_rn(dh, c.hi, -ph);
  pl = __fmaf_rn(dh, c.lo, pl);
  return __fmaf_rn(dl, c.hi, pl);
}

// The weight 2^(ph + pl) of an alive column before its final shift: the mantissa in
// [2^43 (1 - 2^-8), 2^44) and the exponent e <= 0.
__device__ __forceinline__ uint64_t weight_mant(float ph, float pl, const unsigned long long* tab,
                                                int& e) {
  const float magic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer in the low bits
  const float kk = __fmaf_rn(ph, 128.0f, magic);
  const int ki = (int)(__float_as_uint(kk) - 0x4B400000u);
  const float kf = __fsub_rn(kk, magic);
  const float gh = __fmaf_rn(kf, -0.0078125f, ph);  // exact
  const float u = gh + pl;
  // 2^g - 1 in units of 2^-39 (the factors carry them), |.| < 2^31
  const float unit = 549755813888.0f;
  const float ln2h = 0.693147182f * unit, ln2l = -1.90465421e-09f * unit;
  const float t =
      u * u * (0.240226507f * unit + u * (0.0555041087f * unit + u * (0.00961812911f * unit)));
  const float a = __fmul_rn(gh, ln2h);
  float al = __fmaf_rn(gh, ln2h, -a);
  al = __fmaf_rn(gh, ln2l, al);
  al = __fmaf_rn(pl, ln2h, al);
  const float low = __fadd_rn(al + t, magic);  // |al + t| < 2^22
  const int pi = __float2int_rn(a) + (int)(__float_as_uint(low) - 0x4B400000u);
  const unsigned long long tj = tab[ki & 127];
  e = ki >> 7;
  return tj + (uint64_t)(((int64_t)(int32_t)(uint32_t)((tj + 4096) >> 13) * (int64_t)pi) >> 26);
}

// The weight of any logit, without branches: 0 where it is not alive.
__device__ __forceinline__ uint64_t weight_of(float l, float m, const Scale& c,
                                              const unsigned long long* tab) {
  const float ph = lead_log2(l, m, c);
  const bool on = alive(ph);
  const float pl = tail_log2(l, m, c, ph);
  int e;
  const uint64_t mant = weight_mant(on ? ph : 0.0f, on ? pl : 0.0f, tab, e);
  const uint64_t w = (mant + ((1ull << -e) >> 1)) >> -e;
  return on ? w : 0;
}
// An alive column's weight as a float: the hardware's 2^x (2^-22 relative) of the leading part.
__device__ __forceinline__ float weight_float(float l, float m, const Scale& c, float ph) {
  float x;
  asm("ex2.approx.f32 %0, %1;" : "=f"(x) : "f"(ph));
  return __fmaf_rn(x, tail_log2(l, m, c, ph) * 0.693147182f, x);
}

// ceil(f * z) and floor(f * z) for 0 <= f <= 1 in fp32 and z < 2^63, exact.
__device__ __forceinline__ uint64_t mul_frac(float f, uint64_t z, bool up) {
  const uint32_t b = __float_as_uint(f) & 0x7FFFFFFFu;  // -0 counts as 0
  int ex = (int)(b >> 23);
  uint64_t mant = b & 0x7FFFFFu;
  if (ex == 0) ex = 1; else mant |= 0x800000u;
  const int sh = 150 - ex;  // f = mant * 2^-sh, sh >= 23
  const uint64_t lo = mant * z, hi = __umul64hi(mant, z);
  uint64_t q, rest;
  if (sh < 64) {
    q = (lo >> sh) | (hi << (64 - sh));
    rest = lo & ((1ull << sh) - 1);
  } else if (sh < 128) {
    q = sh == 64 ? hi : hi >> (sh - 64);
    rest = lo | (sh == 64 ? 0ull : hi & ((1ull << (sh - 64)) - 1));
  } else {
    q = 0;
    rest = lo | hi;
  }
  return q + ((up && rest != 0) ? 1 : 0);
}

}  // namespace tfd
