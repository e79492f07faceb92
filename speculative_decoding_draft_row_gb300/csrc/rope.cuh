// rope.cuh - qk_norm and RoPE of one head's vector by a warp, shared by the attention kernels.
#pragma once

#include <cmath>

#include "common.cuh"

namespace tfd {

// Each pair's frequency base^(-2i/dim) in turns (1 turn = 2 pi), as a 64-bit binary fraction:
// t_i = frac(base^(-2i/dim) / (2 pi)) * 2^64. For an integer position p, p * t_i mod 2^64 is the
// angle p * base^(-2i/dim) reduced to one turn, exact up to the rounding of t_i (2^-53 relative),
// so the reduction needs no floating-point arithmetic on the device.
template <int D>
struct RopeTurns {
  uint64_t t[D / 2];
};

// The sine and cosine of pair i at position p, of the angle reduced to [-pi, pi).
template <int D>
__device__ __forceinline__ void rope_pair(int p, const RopeTurns<D>& turns, int i, float& sn,
                                          float& cs) {
  const float turn_unit = 1.4629180792671596e-9f;  // 2 pi / 2^32
  const uint64_t ph = (uint64_t)(uint32_t)p * turns.t[i];  // mod 2^64: the reduced angle
  const float red = (float)(int32_t)(ph >> 32) * turn_unit;
  sincosf(red, &sn, &cs);
}

// The same by the hardware's sine and cosine: within 2^-20.5 on [-pi, pi].
template <int D>
__device__ __forceinline__ void rope_pair_fast(int p, const RopeTurns<D>& turns, int i, float& sn,
                                               float& cs) {
  const float turn_unit = 1.4629180792671596e-9f;  // 2 pi / 2^32
  const uint64_t ph = (uint64_t)(uint32_t)p * turns.t[i];
  __sincosf((float)(int32_t)(ph >> 32) * turn_unit, &sn, &cs);
}

// Lane l of a warp holds elements E l .. E l + E - 1 of a vector of D = 32 E elements.
// The sines and cosines of this lane's pairs at position p (lane l holds pairs
// E (l mod 16) .. + E - 1), shared by every head at that position.
template <int D>
__device__ __forceinline__ void rope_sincos(int p, const RopeTurns<D>& turns,
                                            float (&sn)[D / 32], float (&cs)[D / 32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) rope_pair<D>(p, turns, D / 32 * (lane & 15) + j, sn[j], cs[j]);
}

// RMSNorm with gamma.
template <int D>
__device__ __forceinline__ void norm_rows(float (&x)[D / 32], const uint16_t* gamma, float eps) {
  const int lane = threadIdx.x & 31;
  float ss = x[0] * x[0];
#pragma unroll
  for (int j = 1; j < D / 32; ++j) ss += x[j] * x[j];
  ss = warp_sum(ss);
  const float inv = 1.0f / sqrtf(ss / (float)D + eps);
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    const float gm = gamma ? bf16_bits_to_f32(gamma[D / 32 * lane + j]) : 1.0f;
    x[j] = x[j] * inv * gm;
  }
}

// The rotation by the given sines and cosines.
template <int D>
__device__ __forceinline__ void rotate(float (&x)[D / 32], const float (&sn)[D / 32],
                                       const float (&cs)[D / 32]) {
  float other[D / 32];
#pragma unroll
  for (int j = 0; j < D / 32; ++j) other[j] = __shfl_xor_sync(0xffffffffu, x[j], 16);
  const bool first_half = (threadIdx.x & 31) < 16;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    // first half holds a = x[i] (partner b = x[i + D/2]); second half holds b (partner a).
    x[j] = first_half ? (x[j] * cs[j] - other[j] * sn[j]) : (other[j] * sn[j] + x[j] * cs[j]);
  }
}

// RMSNorm with gamma, then the rotation by the given sines and cosines.
template <int D>
__device__ __forceinline__ void norm_rope_sc(float (&x)[D / 32], const uint16_t* gamma, float eps,
                                             const float (&sn)[D / 32], const float (&cs)[D / 32]) {
  norm_rows<D>(x, gamma, eps);
  rotate<D>(x, sn, cs);
}

template <int D>
__device__ __forceinline__ void norm_rope(float (&x)[D / 32], const uint16_t* gamma, float eps,
                                          int p, const RopeTurns<D>& turns) {
  float sn[D / 32], cs[D / 32];
  rope_sincos<D>(p, turns, sn, cs);
  norm_rope_sc<D>(x, gamma, eps, sn, cs);
}

}  // namespace tfd

namespace tfd_host {

// The turn table of a RoPE base, computed in double on the host (kept for the last base used by
// this thread).
template <int D>
const tfd::RopeTurns<D>& rope_turns(float base) {
  thread_local float cached_base = -1.0f;
  thread_local tfd::RopeTurns<D> cached;
  if (cached_base != base) {
    const double two_pi = 6.283185307179586476925286766559;
    for (int i = 0; i < D / 2; ++i) {
      const double f = std::pow((double)base, -2.0 * i / D);
      double turns = f / two_pi;
      turns -= std::floor(turns);
      cached.t[i] = (uint64_t)std::ldexp(turns, 64);
    }
    cached_base = base;
  }
  return cached;
}

}  // namespace tfd_host
