// paged_append.cu - rows of keys and values into their slots of a paged cache: qk_norm and RoPE of the
// keys, then bf16 or E4M3 codes with a scale a vector (largest magnitude / 448).
//
// A sweep bound by its bytes, and for few rows by latency: a warp takes some heads of a row, 16 bytes a
// lane, loads its next vectors (and their slot) before it uses these, and forms a position's sines and
// cosines once, a pair or two a lane, shared through shared memory. 8193 rows of 8 heads of 128 in bf16 14.8 us,
// 0.67 of the copy rate (one item a warp, loads after the slot is known: 18.6); in E4M3 29.8, 0.25, bound by its sixteen
// exact divisions a lane for a pair of vectors; one draft step 2.6 us.
#include "paged.cuh"

namespace {

using namespace tfd;

constexpr int kT = 256;

// Steps of an item (2 heads of 128 or 4 of 64 each), and blocks of an SM that registers allow for it.
constexpr int blocks_of(int iter) { return iter == 1 ? 3 : 2; }

template <int D>
struct Args {
  const uint16_t* k_rows;
  const uint16_t* v_rows;
  int64_t ldk, ldv;
  const int32_t* slots;
  const int32_t* pos;
  const uint16_t* gamma;
  tfd_kv_pages c;
  int32_t* dev_status;
  int rows, groups, qk;
  float eps;
  RopeTurns<D> turns;
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// One vector's codes and scale, 8 elements a lane of L.
template <int L>
__device__ __forceinline__ void put_codes(const float (&x)[8], uint8_t* to, float* scale, bool one) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
#pragma unroll
  for (int m = L / 2; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  const float s = __fdiv_rn(amax, 448.0f);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = s > 0.0f ? __fdiv_rn(x[4 * i + e], s) : x[4 * i + e];
    w[i] = e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16);
  }
  if (to) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
  if (to && one) *scale = s;
}

// A warp's share of a row into its slot.
template <int D, bool kF8, int kIter>
__device__ __forceinline__ void write_item(const Args<D>& a, const RopeTurns<D>& turns, float2* turn, int64_t w,
                                           int slot, int p, const uint4 (&kr)[kIter], const uint4 (&vr)[kIter],
                                           const float (&gm)[8]) {
  constexpr int L = D / 8, kPer = 32 / L;  // lanes of a vector, vectors of a step
  const int lane = threadIdx.x & 31, l = lane % L;
  const int h0 = (int)(w % a.groups) * (kIter * kPer) + lane / L;
  if (slot == -1) return;
  if (slot < 0 || slot >= a.c.pages * a.c.page_size || p < 0) {
    if (lane == 0) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
    return;
  }
  float sn[8], cs[8];
  if (a.qk & TFD_QK_ROPE) {
    __syncwarp();  // the last item's are done with
#pragma unroll
    for (int i = lane; i < D / 2; i += 32) rope_pair_fast<D>(p, turns, i, turn[i].y, turn[i].x);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float4 t = *reinterpret_cast<const float4*>(&turn[8 * (l % (L / 2)) + j]);
      cs[j] = t.x, sn[j] = t.y, cs[j + 1] = t.z, sn[j + 1] = t.w;
    }
  }
  const int page = slot / a.c.page_size, at = slot - page * a.c.page_size;
  const int64_t base = page * a.c.page_stride + at * a.c.token_stride + 8 * l;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int h = h0 + i * kPer;
    const bool in = h < a.c.heads;
    const uint32_t kw[4] = {kr[i].x, kr[i].y, kr[i].z, kr[i].w};
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[2 * j] = bf16_lo(kw[j]), x[2 * j + 1] = bf16_hi(kw[j]);
    if (a.qk & TFD_QK_NORM) {
      float ss = x[0] * x[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
      for (int m = L / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float inv = 1.0f / sqrtf(ss / (float)D + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * gm[j];
    }
    if (a.qk & TFD_QK_ROPE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float other = __shfl_xor_sync(0xffffffffu, x[j], L / 2);
        x[j] = l < L / 2 ? x[j] * cs[j] - other * sn[j] : other * sn[j] + x[j] * cs[j];
      }
    }
    const int64_t to = base + h * a.c.head_stride;
    if (kF8) {
      const int64_t sc = ((int64_t)page * a.c.heads + h) * a.c.page_size + at;
      put_codes<L>(x, in ? (uint8_t*)a.c.k + to : nullptr, a.c.k_scales + sc, l == 0);
      const uint32_t vw[4] = {vr[i].x, vr[i].y, vr[i].z, vr[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) x[2 * j] = bf16_lo(vw[j]), x[2 * j + 1] = bf16_hi(vw[j]);
      put_codes<L>(x, in ? (uint8_t*)a.c.v + to : nullptr, a.c.v_scales + sc, l == 0);
    } else if (in) {
      uint4 o = kr[i];
      if (a.qk) {
        uint32_t* ow = &o.x;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ow[j] = (uint32_t)f32_to_bf16_bits(x[2 * j]) |
                  ((uint32_t)f32_to_bf16_bits(x[2 * j + 1]) << 16);
      }
      *reinterpret_cast<uint4*>((uint16_t*)a.c.k + to) = o;
      *reinterpret_cast<uint4*>((uint16_t*)a.c.v + to) = vr[i];
    }
  }
}

template <int D, bool kF8, int kIter>
__global__ void __launch_bounds__(kT, blocks_of(kIter)) paged_append_kernel(const Args<D> a) {
  constexpr int L = D / 8, kPer = 32 / L;  // lanes of a vector, vectors of a step
  __shared__ __align__(16) float2 turn[kT / 32][D / 2];
  // the pairs' frequencies: as an argument each lane's would be fetched after the other's, every time
  __shared__ RopeTurns<D> turns;
  if (threadIdx.x < D / 2) turns.t[threadIdx.x] = a.turns.t[threadIdx.x];
  __syncthreads();
  tfd_host::after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % L;
  float gm[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    gm[j] = a.gamma && (a.qk & TFD_QK_NORM) ? bf16_bits_to_f32(a.gamma[8 * l + j]) : 1.0f;
  // an item: the heads of a row that a warp takes; the next one's vectors are loaded before this one's are used
  const int64_t items = (int64_t)a.rows * a.groups, step = (int64_t)gridDim.x * (kT / 32);
  uint4 kr[kIter], vr[kIter];
  int slot = -1, p = 0;
  auto load = [&](int64_t w) {
    if (w >= items) return;
    const int row = (int)(w / a.groups), h0 = (int)(w - (int64_t)row * a.groups) * (kIter * kPer) + lane / L;
    slot = a.slots[row];
    p = a.qk & TFD_QK_ROPE ? a.pos[row] : 0;
    const uint16_t* kp = a.k_rows + row * a.ldk + (int64_t)h0 * D + 8 * l;
    const uint16_t* vp = a.v_rows + row * a.ldv + (int64_t)h0 * D + 8 * l;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const bool in = h0 + i * kPer < a.c.heads;
      kr[i] = in ? *reinterpret_cast<const uint4*>(kp + i * kPer * D) : make_uint4(0u, 0u, 0u, 0u);
      vr[i] = in ? *reinterpret_cast<const uint4*>(vp + i * kPer * D) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  int64_t w = (int64_t)blockIdx.x * (kT / 32) + warp;
  load(w);
  for (; w < items; w += step) {
    uint4 k_now[kIter], v_now[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) k_now[i] = kr[i], v_now[i] = vr[i];
    const int slot_now = slot, p_now = p;
    load(w + step);
    write_item<D, kF8, kIter>(a, turns, turn[warp], w, slot_now, p_now, k_now, v_now, gm);
  }
}

template <int D, bool kF8, int kIter>
tfd_status launch_items(Args<D>& a, int dev, int sms, cudaStream_t stream) {
  constexpr int heads = kIter * 32 / (D / 8);  // of an item
  a.groups = (a.c.heads + heads - 1) / heads;
  const int64_t blocks = ((int64_t)a.rows * a.groups + kT / 32 - 1) / (kT / 32);
  return tfd_host::launch_clusters<paged_append_kernel<D, kF8, kIter>>(
      a, dev, std::min(blocks, (int64_t)sms * blocks_of(kIter)), 1, kT, 0, 0, stream);
}

// Items of one step while there is a warp for each at once (288 rows of 8 heads 3.9 us, with four steps 7.8);
// beyond, four steps share a row's sines and cosines and keep more loads in flight (8193 rows 14.8 us, with one
// step 18.2).
template <int D, bool kF8>
tfd_status launch(Args<D>& a, float rope_base, cudaStream_t stream) {
  if (a.qk & TFD_QK_ROPE) a.turns = tfd_host::rope_turns<D>(rope_base);
  int dev = 0;
  const int sms = std::max(1, tfd_host::device_sms(dev));
  const int64_t single = (int64_t)a.rows * ((a.c.heads * (D / 8) + 31) / 32);
  return single <= (int64_t)sms * blocks_of(1) * (kT / 32) ? launch_items<D, kF8, 1>(a, dev, sms, stream)
                                                           : launch_items<D, kF8, 4>(a, dev, sms, stream);
}

template <int D>
tfd_status launch_dim(const void* k_rows, int64_t ldk, const void* v_rows, int64_t ldv,
                      const int32_t* slots, const int32_t* pos, int rows, int qk,
                      const void* k_gamma, float eps, float rope_base, const tfd_kv_pages& c,
                      int32_t* dev_status, cudaStream_t stream) {
  Args<D> a = {(const uint16_t*)k_rows, (const uint16_t*)v_rows, ldk, ldv, slots, pos,
               (const uint16_t*)k_gamma, c, dev_status, rows, 0, qk, eps, {}};
  return c.fmt == TFD_KV_E4M3 ? launch<D, true>(a, rope_base, stream)
                              : launch<D, false>(a, rope_base, stream);
}

}  // namespace

extern "C" tfd_status tfd_paged_append(const void* k_rows, int64_t ldk, const void* v_rows,
                                       int64_t ldv, const int32_t* slots, const int32_t* pos,
                                       int rows, int qk, const void* k_gamma, float eps,
                                       float rope_base, const tfd_kv_pages* cache,
                                       int32_t* dev_status, void* stream) {
  using tfd_host::aligned;
  if (!k_rows || !v_rows || !slots || rows < 1) return TFD_ERR_INVALID;
  const tfd_status st = tfd_paged::check_cache(cache);
  if (st != TFD_OK) return st;
  const tfd_kv_pages& c = *cache;
  if (!tfd_paged::check_qk(qk, eps, rope_base) || ((qk & TFD_QK_ROPE) && !pos))
    return TFD_ERR_INVALID;
  const int64_t width = (int64_t)c.heads * c.dim;
  if (ldk < width || ldv < width || ldk % 8 || ldv % 8) return TFD_ERR_INVALID;
  if ((int64_t)rows * c.heads > 2147483647 || ldk > ((int64_t)1 << 30) || ldv > ((int64_t)1 << 30))
    return TFD_ERR_UNSUPPORTED;
  if (!aligned(k_rows, 16) || !aligned(v_rows, 16) || !aligned(slots, 4) || !aligned(pos, 4) ||
      !aligned(k_gamma, 2) || !aligned(dev_status, 4))
    return TFD_ERR_INVALID;
  using tfd_paged::overlaps_cache;
  if (overlaps_cache(c, k_rows, ((int64_t)(rows - 1) * ldk + width) * 2) ||
      overlaps_cache(c, v_rows, ((int64_t)(rows - 1) * ldv + width) * 2) ||
      overlaps_cache(c, slots, rows * 4ll) || overlaps_cache(c, pos, pos ? rows * 4ll : 0) ||
      overlaps_cache(c, k_gamma, k_gamma ? c.dim * 2 : 0) || overlaps_cache(c, dev_status, 4))
    return TFD_ERR_INVALID;
  cudaStream_t s = tfd_host::as_stream(stream);
  return c.dim == 64 ? launch_dim<64>(k_rows, ldk, v_rows, ldv, slots, pos, rows, qk, k_gamma, eps,
                                      rope_base, c, dev_status, s)
                     : launch_dim<128>(k_rows, ldk, v_rows, ldv, slots, pos, rows, qk, k_gamma,
                                       eps, rope_base, c, dev_status, s);
}
