// lora.cuh - what the adapter kernels share: their arguments, and the search for a block's tile of rows.
#pragma once

#include "launch.cuh"

namespace tfd_adapters {

using namespace tfd;

constexpr int kT = 256;
constexpr int kW = kT / 32;
constexpr int kMaxAdapters = 4096;
constexpr int kSmallRows = 256;  // up to here one thread a row groups the rows

struct Args {
  const __nv_bfloat16* x;
  int64_t ldx;
  const __nv_bfloat16* a;
  const __nv_bfloat16* b;
  const int32_t* ids;
  const float* scales;
  const char* base;
  char* y;
  int64_t ldb, ldy;
  int32_t* dev_status;
  int rows, k, n, rank, n_adapters, splits;
  int smem;  // bytes of shared memory that the tile search may use
  bool f32, vec;
};

// Takes the leading bf16 part off v, in which it stays within bf16's range: parts taken one after the
// other add up to a finite v (24 bits in three). An infinity or NaN goes whole into its first part,
// with zeros behind it: as a difference, inf - inf, the rest would make NaN of an infinite product.
__device__ __forceinline__ __nv_bfloat16 take_part(float& v) {
  const float most = __uint_as_float(0x7F7F0000u);  // bf16's largest
  const bool finite = fabsf(v) < INFINITY;
  const __nv_bfloat16 x = __float2bfloat16_rn(finite ? fminf(fmaxf(v, -most), most) : v);
  v = finite ? v - __bfloat162float(x) : 0.0f;
  return x;
}

// Which adapter (n_adapters = none) and which rows tile `t` has; 0 rows when there is no such tile.
template <int TM, int T = kT>
__device__ int find_tile(const Args& a, int t, int32_t* rows_out, int32_t* cnt, int& key) {
  __shared__ int s_key, s_first, s_n, s_warp[T / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_n = 0;
  auto key_of = [&](int r) {
    const int id = a.ids[r];
    if (id >= 0 && id < a.n_adapters) return id;
    if (id != -1) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
    return a.n_adapters;
  };
  if (a.rows <= kSmallRows) {
    int mine = -1, c = 0;
    if (tid < a.rows) cnt[tid] = mine = key_of(tid);
    __syncthreads();
    for (int j = 0; j < tid && tid < a.rows; ++j) c += cnt[j] == mine;
    const bool first = tid < a.rows && c % TM == 0;
    const unsigned bal = __ballot_sync(0xffffffffu, first);
    if (lane == 0) s_warp[warp] = __popc(bal);
    __syncthreads();
    int no = __popc(bal & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) no += s_warp[w];
    if (first && no == t) {
      s_key = mine;
      s_first = c;
      s_n = 1;
    }
    __syncthreads();
    if (s_n == 0) return 0;
    key = s_key;
    const int at = c - s_first;
    const bool member = tid < a.rows && mine == key && at >= 0 && at < TM;
    if (member) rows_out[at] = tid;
    const int n = __syncthreads_count(member);
    return n;
  }
  // counts of every adapter, the tiles before and of each, then the members in row order; the keys
  // stay in shared memory where they fit
  for (int i = tid; i <= a.n_adapters; i += T) cnt[i] = 0;
  uint16_t* keys = reinterpret_cast<uint16_t*>(cnt + a.n_adapters + 1);
  const bool kept = a.rows <= (a.smem - 4 * (a.n_adapters + 1)) / 2;
  __syncthreads();
#pragma unroll 1
  for (int r0 = 0; r0 < a.rows; r0 += 4 * T) {
    int id[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // the loads first
      const int r = r0 + q * T + tid;
      id[q] = r < a.rows ? a.ids[r] : -2;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = r0 + q * T + tid;
      const bool in = r < a.rows;
      const bool good = id[q] >= 0 && id[q] < a.n_adapters;
      if (in && !good && id[q] != -1) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
      const int kk = in ? (good ? id[q] : a.n_adapters) : -1;
      if (kept && in) keys[r] = (uint16_t)kk;
      int same;
      __match_all_sync(0xffffffffu, kk, &same);
      if (same) {  // a prompt's rows adjoin
        if (kk >= 0 && lane == 0) atomicAdd(&cnt[kk], 32);
      } else if (kk >= 0) {
        atomicAdd(&cnt[kk], 1);
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    int before = 0;
    for (int i0 = 0; i0 <= a.n_adapters; i0 += 32) {
      const int i = i0 + lane;
      const int m = i <= a.n_adapters ? (cnt[i] + TM - 1) / TM : 0;
      int incl = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (t >= before + incl - m && t < before + incl) {
        s_key = i;
        s_first = (t - (before + incl - m)) * TM;
        s_n = min(TM, cnt[i] - s_first);
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  __syncthreads();
  const int n = s_n;
  if (n == 0) return 0;
  key = s_key;
  const int per = (a.rows + T - 1) / T, r0 = tid * per, r1 = min(a.rows, r0 + per);
  auto is_mine = [&](int r) {
    if (kept) return (int)keys[r] == key;
    const int id = a.ids[r];
    return (id >= 0 && id < a.n_adapters ? id : a.n_adapters) == key;
  };
  int c = 0;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) c += is_mine(r);
  int incl = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int at = incl - c - s_first;
  for (int w = 0; w < warp; ++w) at += s_warp[w];
  if (c > 0 && at < TM && at + c > 0) {
    for (int r = r0; r < r1; ++r) {
      if (!is_mine(r)) continue;
      if (at >= 0 && at < TM) rows_out[at] = r;
      ++at;
    }
  }
  __syncthreads();
  return n;
}

// The tensor-memory form for many rows an adapter (lora_tc.cu). *taken says whether it applies.
tfd_status launch_tc(Args a, int dev, cudaStream_t stream, bool* taken);

}  // namespace tfd_adapters
