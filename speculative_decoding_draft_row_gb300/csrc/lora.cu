// lora.cu - low-rank adapters of many requests at once: y_r = base_r + s_a B_a (A_a x_r), a the
// adapter of row r, for one decode row up to whole prompts, in one launch without a workspace.
//
// Rows are grouped by adapter into tiles of up to TM rows, so an adapter used by many rows is read
// once a tile. Every block derives its tile from the ids itself (a count per adapter, then the
// members of its own tile): a few thousand ids cost less than another launch.
//
// A thread-block cluster takes a tile. Shrink: h = A x over the rank x TM outputs, k split over the
// cluster's blocks and their warps; both operands go from global memory straight to the registers
// of warp-level MMAs (m16n8k16, A the 16 ranks, x the 8 rows), since within a tile every weight and
// every activation is used by one warp only. The k order is permuted alike for both so that a
// thread's 16 contiguous bytes are its operands. The partial sums are added in a fixed order, over
// the warps and, through distributed shared memory, over the blocks: every block then has all of h.
// Expand: each block takes a range of the n outputs in steps of 32 a warp; h is the MMA's row
// operand, split into bf16 parts that add up to it (below), and B's rows its columns, dealt so that
// a thread holds 8 contiguous outputs of a row: 16-byte loads of the base and stores of y. The
// first step's rows of B are in flight while h is reduced.
//
// h stays in fp32 and enters the MMAs as two (bf16 outputs: 2^-17 relative, under a 2^-9 rounding) or
// three (fp32 outputs: all 24 bits) bf16 parts, whose products are exact in the fp32 accumulators.
//
// Bound by latency: one row 4096 to 4096 at rank 16 takes 5.3 us, 16 rows 11008 to 4096 of eight
// adapters at rank 32 7.4, 16 rows over a 163840-row head of four adapters at rank 16 15.3 (42 MB,
// 0.41 of the copy rate). L2 prefetches of what the expand reads made them slower by 0.6 to 2 us.
#include <cooperative_groups.h>

#include "lora.cuh"

namespace {

using namespace tfd;
using namespace tfd_adapters;
namespace cg = cooperative_groups;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

// Blocks an SM. The expand waits for what it reads: three of the smallest form, whose 80 registers hold
// without a spill, keep more of it in flight (16 rows over a 163840-row head at rank 16: 15.5 us, two
// 16.9; four of 64 registers spill, 19.2).
template <int RT, int NT>
constexpr int kBlocks = RT == 1 && NT == 1 ? 3 : 2;

// RT: 16-rank tiles (rank <= 16 RT); NT: 8-row tiles of x (TM = 8 NT).
template <int RT, int NT>
__global__ void __launch_bounds__(kT, kBlocks<RT, NT>) lora_kernel(const Args a) {
  constexpr int TM = 8 * NT, R = 16 * RT, RP = R + 4;  // RP: partial sums without bank conflicts
  constexpr int MT = (TM + 15) / 16, HT = 16 * MT;     // row tiles of the expand
  constexpr int KP = RT == 1 ? 1 : RT / 2;             // 16-byte (RT 1: 8-byte) pieces of a B row
  constexpr int HP = R + 8;
  constexpr bool AHEAD = RT <= 2;                      // two steps' rows of B fit the registers
  extern __shared__ __align__(16) unsigned char smem[];
  float* part = reinterpret_cast<float*>(smem);                  // [kW][TM][RP]
  float* mine = part + kW * TM * RP;                             // [TM][RP], read by the cluster
  __nv_bfloat16* hs = reinterpret_cast<__nv_bfloat16*>(mine + TM * RP);  // [3][HT][HP]
  __shared__ int32_t tile_rows[TM];
  tfd_host::after_previous();
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank_c = (int)cl.block_rank();
  const int unit = blockIdx.x / C, tile = unit / a.splits, split = unit % a.splits;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  int key = 0;
  const int m = find_tile<TM>(a, tile, tile_rows, reinterpret_cast<int32_t*>(smem), key);
  if (m == 0) return;  // all blocks of the cluster alike
  const bool none = key == a.n_adapters;
  if (none && a.base == a.y) return;

  // this block's share of the outputs, in steps of 32
  const int steps = (a.n + 31) / 32, parts = C * a.splits, part_no = split * C + rank_c;
  const int s0 = (int)((int64_t)steps * part_no / parts);
  const int s1 = (int)((int64_t)steps * (part_no + 1) / parts);
  const __nv_bfloat16* bw = a.b + (int64_t)(none ? 0 : key) * a.n * a.rank;

  // rows of B of step s: tile j, column g -> output 32 s + 8 (g / 2) + 2 j + g % 2
  auto load_b = [&](int s, uint4 (&w)[4][KP]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int o = s * 32 + (g >> 1) * 8 + 2 * j + (g & 1);
      const __nv_bfloat16* row = bw + (int64_t)o * a.rank;
#pragma unroll
      for (int q = 0; q < KP; ++q) {
        w[j][q] = zero4();
        if (RT == 1) {
          if (o < a.n && 4 * t < a.rank) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + 4 * t));
            w[j][q].x = v.x;
            w[j][q].y = v.y;
          }
        } else if (o < a.n && 32 * q + 8 * t < a.rank) {
          w[j][q] = __ldg(reinterpret_cast<const uint4*>(row + 32 * q + 8 * t));
        }
      }
    }
  };

  uint4 wb[4][KP];
  if (!none) {
    // ---- shrink -------------------------------------------------------------------------------
    const int blocks = (a.k + 31) / 32, slots = C * kW, slot = rank_c * kW + warp;
    const int b0 = (int)((int64_t)blocks * slot / slots);
    const int b1 = (int)((int64_t)blocks * (slot + 1) / slots);
    const __nv_bfloat16* aw = a.a + ((int64_t)key * a.rank + g) * a.k + 8 * t;
    const __nv_bfloat16* xr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int i = 8 * j + g;  // rows past the tile's last repeat it; their sums are not used
      xr[j] = a.x + (int64_t)tile_rows[min(i, m - 1)] * a.ldx + 8 * t;
    }
    float acc[RT][NT][4] = {};
#pragma unroll 2
    for (int b = b0; b < b1; ++b) {
      const int k0 = b * 32;
      const bool in = k0 + 8 * t < a.k;
      uint4 av[RT][2], xv[NT];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          av[i][h] = in && 16 * i + 8 * h + g < a.rank
                         ? __ldg(reinterpret_cast<const uint4*>(aw + (int64_t)(16 * i + 8 * h) * a.k + k0))
                         : zero4();
#pragma unroll
      for (int j = 0; j < NT; ++j)
        xv[j] = in ? __ldg(reinterpret_cast<const uint4*>(xr[j] + k0)) : zero4();
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma(acc[i][j], av[i][0].x, av[i][1].x, av[i][0].y, av[i][1].y, xv[j].x, xv[j].y);
          mma(acc[i][j], av[i][0].z, av[i][1].z, av[i][0].w, av[i][1].w, xv[j].z, xv[j].w);
        }
    }
    if (s0 + warp < s1) load_b(s0 + warp, wb);  // in flight while h is reduced
    __syncthreads();                            // the tile search's counts are done with
    float* p = part + warp * TM * RP;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          p[(8 * j + 2 * t + (e & 1)) * RP + 16 * i + g + 8 * (e >> 1)] = acc[i][j][e];
    __syncthreads();
    for (int i = tid; i < TM * R; i += kT) {
      const int o = (i / R) * RP + i % R;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kW; ++w) v += part[w * TM * RP + o];
      mine[o] = v;
    }
    cl.sync();
    const float scale = a.scales ? a.scales[key] : 1.0f;
    for (int i = tid; i < HT * R; i += kT) {
      const int row = i / R, o = row * RP + i % R;
      float v = 0.0f;
      if (row < TM)
        for (int c = 0; c < C; ++c) v += cl.map_shared_rank(mine, c)[o];
      v = i % R < a.rank ? v * scale : 0.0f;  // past the adapter's ranks 0 x inf would be NaN
      hs[row * HP + i % R] = take_part(v);
      hs[(HT + row) * HP + i % R] = take_part(v);
      if (a.f32) hs[(2 * HT + row) * HP + i % R] = take_part(v);
    }
    cl.barrier_arrive();  // this block has read the others' sums
    __syncthreads();
  }

  // ---- expand -----------------------------------------------------------------------------------
  // The next step's rows of B (while two steps' fit the registers) and, for one row tile, this step's
  // base are on their way during the MMAs: the loop is bound by the latency of what it reads (16 rows
  // over a 163840-row head at rank 16: 23.2 us without, 19.0 with).
  const int parts_h = a.f32 ? 3 : 2;
  for (int s = s0 + warp; s < s1; s += kW) {
    const int o = s * 32 + 8 * t;
    uint4 wn[AHEAD ? 4 : 1][KP];
    if constexpr (AHEAD) {
      if (!none && s + kW < s1) load_b(s + kW, wn);
    } else {
      if (!none && s != s0 + warp) load_b(s, wb);
    }
    const bool whole = a.vec && o + 8 <= a.n;
    uint4 br[2][2];
    if (MT == 1) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int slot = 8 * h + g;
        br[h][0] = br[h][1] = zero4();
        if (whole && a.base && slot < m) {
          const char* bp = a.base + ((int64_t)tile_rows[slot] * a.ldb + o) * (a.f32 ? 4 : 2);
          br[h][0] = *reinterpret_cast<const uint4*>(bp);
          if (a.f32) br[h][1] = *reinterpret_cast<const uint4*>(bp + 16);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      float acc[4][4] = {};
      if (!none) {
#pragma unroll
        for (int q = 0; q < (RT == 1 ? 1 : 2 * KP); ++q) {
          // 16 ranks: RT 1: 4t .. 4t+3; else half q % 2 of the thread's 8
          const int col = RT == 1 ? 4 * t : 32 * (q >> 1) + 8 * t + 4 * (q & 1);
          for (int h = 0; h < parts_h; ++h) {
            const uint2 u = *reinterpret_cast<const uint2*>(hs + (h * HT + 16 * i + g) * HP + col);
            const uint2 v =
                *reinterpret_cast<const uint2*>(hs + (h * HT + 16 * i + 8 + g) * HP + col);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 w = wb[j][q >> 1];
              mma(acc[j], u.x, v.x, u.y, v.y, (q & 1) ? w.z : w.x, (q & 1) ? w.w : w.y);
            }
          }
        }
      }
      if (o >= a.n) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int slot = 16 * i + 8 * h + g;
        if (slot >= m) continue;
        const int64_t row = tile_rows[slot];
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = acc[j][2 * h];
          v[2 * j + 1] = acc[j][2 * h + 1];
        }
        const char* bp = a.base + (row * a.ldb + o) * (a.f32 ? 4 : 2);
        char* yp = a.y + (row * a.ldy + o) * (a.f32 ? 4 : 2);
        if (whole) {
          uint4 r0 = br[h][0], r1 = br[h][1];
          if (MT > 1) {
            r0 = r1 = zero4();
            if (a.base) {
              r0 = *reinterpret_cast<const uint4*>(bp);
              if (a.f32) r1 = *reinterpret_cast<const uint4*>(bp + 16);
            }
          }
          if (a.f32) {
            *reinterpret_cast<float4*>(yp) =
                make_float4(__uint_as_float(r0.x) + v[0], __uint_as_float(r0.y) + v[1],
                            __uint_as_float(r0.z) + v[2], __uint_as_float(r0.w) + v[3]);
            *reinterpret_cast<float4*>(yp + 16) =
                make_float4(__uint_as_float(r1.x) + v[4], __uint_as_float(r1.y) + v[5],
                            __uint_as_float(r1.z) + v[6], __uint_as_float(r1.w) + v[7]);
          } else {
            uint32_t* w = &r0.x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = (uint32_t)f32_to_bf16_bits(bf16_lo(w[e]) + v[2 * e]) |
                     ((uint32_t)f32_to_bf16_bits(bf16_hi(w[e]) + v[2 * e + 1]) << 16);
            *reinterpret_cast<uint4*>(yp) = r0;
          }
        } else if (a.f32) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (o + e < a.n)
              reinterpret_cast<float*>(yp)[e] =
                  (a.base ? reinterpret_cast<const float*>(bp)[e] : 0.0f) + v[e];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (o + e < a.n)
              reinterpret_cast<uint16_t*>(yp)[e] = f32_to_bf16_bits(
                  (a.base ? bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(bp)[e]) : 0.0f) +
                  v[e]);
        }
      }
    }
    if constexpr (AHEAD) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < KP; ++q) wb[j][q] = wn[j][q];
    }
  }
  if (!none) cl.barrier_wait();  // the others have read this block's sums
}

template <int RT, int NT>
tfd_status launch(Args a, int dev, int c, int64_t units, cudaStream_t stream) {
  constexpr int TM = 8 * NT, R = 16 * RT, RP = R + 4, HT = (TM + 15) / 16 * 16;
  size_t smem = (size_t)(kW + 1) * TM * RP * 4 + (size_t)3 * HT * (R + 8) * 2;
  const size_t counts = (size_t)4 * (a.rows <= kSmallRows ? kSmallRows : a.n_adapters + 1);
  if (smem < counts) smem = counts;
  a.smem = (int)smem;
  return tfd_host::launch_clusters<lora_kernel<RT, NT>>(a, dev, units, c, kT, smem, 112 * 1024, stream);
}

}  // namespace

extern "C" tfd_status tfd_lora(const void* x, int rows, int64_t k, int64_t ldx, const void* a_w,
                               const void* b_w, int n_adapters, int rank, int64_t n,
                               const int32_t* adapter_ids, const float* scales, int out_mode,
                               const void* base, int64_t ldb, void* y, int64_t ldy,
                               int32_t* dev_status, void* stream) {
  using tfd_host::aligned;
  if (!x || !a_w || !b_w || !adapter_ids || !y) return TFD_ERR_INVALID;
  if (out_mode != TFD_OUT_F32 && out_mode != TFD_OUT_BF16) return TFD_ERR_INVALID;
  if (rows < 1 || k < 8 || k % 8 || n < 1 || n_adapters < 1 || rank < 8 || rank % 8)
    return TFD_ERR_INVALID;
  if (ldx < k || ldx % 8 || ldy < n || (base && ldb < n)) return TFD_ERR_INVALID;
  if (rank > TFD_MAX_RANK || n_adapters > kMaxAdapters || k > (1 << 24) || n > (1 << 24) ||
      rows > TFD_MAX_LORA_ROWS)
    return TFD_ERR_UNSUPPORTED;
  const int es = out_mode == TFD_OUT_F32 ? 4 : 2;
  if (!aligned(x, 16) || !aligned(a_w, 16) || !aligned(b_w, 16) || !aligned(y, es) ||
      !aligned(base, es) || !aligned(adapter_ids, 4) || !aligned(scales, 4) ||
      !aligned(dev_status, 4))
    return TFD_ERR_INVALID;
  using tfd_host::overlap;
  const int64_t ybytes = (((int64_t)rows - 1) * ldy + n) * es;
  if (overlap(y, ybytes, x, (((int64_t)rows - 1) * ldx + k) * 2) ||
      overlap(y, ybytes, a_w, (int64_t)n_adapters * rank * k * 2) ||
      overlap(y, ybytes, b_w, (int64_t)n_adapters * rank * n * 2) ||
      overlap(y, ybytes, adapter_ids, (int64_t)rows * 4) ||
      overlap(y, ybytes, scales, (int64_t)n_adapters * 4))
    return TFD_ERR_INVALID;
  if (base && !(base == y && ldb == ldy) &&
      overlap(y, ybytes, base, (((int64_t)rows - 1) * ldb + n) * es))
    return TFD_ERR_INVALID;

  const bool vec = aligned(y, 16) && ldy * es % 16 == 0 &&
                   (!base || (aligned(base, 16) && ldb * es % 16 == 0));
  // rows of a tile: what one adapter is likely to have, within the accumulators' registers
  const int rt = rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8;
  const int each = (rows + n_adapters - 1) / n_adapters;
  int nt = each <= 8 ? 1 : each <= 32 ? 2 : 16 / rt;
  if (nt > 8) nt = 8;
  const int tm = 8 * nt;
  const int64_t bound = (int64_t)rows / tm + n_adapters + 1;
  const int64_t tiles = bound < rows ? bound : rows;
  // blocks: as many as fit the SMs once, a cluster's share of k and n at least 32 a warp
  int64_t likely = (rows + tm - 1) / tm;
  if (likely < n_adapters) likely = n_adapters < rows ? n_adapters : rows;
  int dev = 0;
  const int sms = tfd_host::device_sms(dev);
  const int64_t wide = k > n ? k : n;
  int c = 1, splits = 1;
  while (c < 8 && likely * c * 2 <= 2 * sms && wide / (c * 2) >= 32 * kW) c *= 2;
  const size_t room = 16 * 1024;
  auto at_once = [&](int blocks) {
    return rt == 1 && nt == 1
               ? tfd_host::clusters_at_once<lora_kernel<1, 1>>(dev, blocks, kT, room)
               : tfd_host::clusters_at_once<lora_kernel<4, 1>>(dev, blocks, kT, room);
  };
  while (c > 1 && at_once(c) == 0) c /= 2;  // no cluster of that size can be placed
  if (c == 8) {  // within one round of clusters
    while (likely * (splits + 1) <= at_once(c) && n / (c * (splits + 1)) >= 32 * kW &&
           n / splits >= 2 * k)
      ++splits;
  }
  Args a = {(const __nv_bfloat16*)x, ldx, (const __nv_bfloat16*)a_w, (const __nv_bfloat16*)b_w,
            adapter_ids, scales, (const char*)base, (char*)y, ldb, ldy, dev_status, rows, (int)k,
            (int)n, rank, n_adapters, splits, 0, es == 4, vec};
  cudaStream_t st = tfd_host::as_stream(stream);
  bool taken = false;
  const tfd_status tc = launch_tc(a, dev, st, &taken);
  if (taken || tc != TFD_OK) return tc;
  const int64_t units = tiles * splits;
  if (units * c > 0x7fffffff) return TFD_ERR_UNSUPPORTED;
#define TFD_LORA_CASE(RT, NT) \
  if (rt == RT && nt == NT) return launch<RT, NT>(a, dev, c, units, st);
  TFD_LORA_CASE(1, 1) TFD_LORA_CASE(1, 2) TFD_LORA_CASE(1, 8)
  TFD_LORA_CASE(2, 1) TFD_LORA_CASE(2, 2) TFD_LORA_CASE(2, 8)
  TFD_LORA_CASE(4, 1) TFD_LORA_CASE(4, 2) TFD_LORA_CASE(4, 4)
  TFD_LORA_CASE(8, 1) TFD_LORA_CASE(8, 2)
#undef TFD_LORA_CASE
  return TFD_ERR_UNSUPPORTED;
}
