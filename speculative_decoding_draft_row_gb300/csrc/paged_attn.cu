// paged_attn.cu - attention of a request's new rows over its tokens in a paged key-value cache, one
// pass with a running maximum and sum, split over the cache's length and joined.
//
// Work. A unit is one request, one key head, and up to 16 MT of its (row, query head) pairs, which share
// every key and value read. The units' tokens, cut into tiles, form one line over all requests; each
// block takes an equal stretch of it, found by a prefix sum over the requests that every block forms
// for itself, so lengths can stay on the GPU and long requests spread over all SMs. A stretch that
// covers a unit writes its rows; the others leave (maximum, sum, weighted values) in the workspace, and
// the block that arrives last adds the unit's pieces in their order along the line (a counter for each block
// in which a unit begins; nobody waits, and the sums' order does not depend on who is last).
//
// A warp takes a slice of 16 or 32 tokens of each tile through a ring of its own in shared memory
// (cp.async, 16 bytes a lane, 128-byte rows swizzled for ldmatrix), so no barrier stands in the loop. Scores and
// values are warp-level MMAs with fp32 accumulators: at 16 rows a unit they need a third of the tensor
// rate that the bytes leave, so q' and the probabilities go in as two bf16 parts each (2^-17 of their value)
// instead of being rounded. E4M3 keys are widened to f16 (exact) against q' over a power of two in two
// f16 parts; E4M3 values to bf16 (exact), their scales in the probabilities, which keep fp32's range.
//
// What a row does not see gets a score of -inf and a weight of zero; tokens past the last and on bad
// pages are zero-filled. In slices with hidden tokens whose values hold an infinity or NaN (0 times
// which would be NaN) the weights are multiplied by hand, only where the row sees the token.
#include <cuda_fp16.h>

#include "paged.cuh"

namespace {

using namespace tfd;

constexpr int kT = 128;
constexpr int kW = kT / 32;
constexpr int kStages = 3;
constexpr int kPerSm = 2;
constexpr int kMostTokens = 0x7fffffff - 1024;  // of a request: a tile behind them is still an int
constexpr int kMaxBlocks = 304;  // blocks of a launch at most: 2 an SM of 152

template <int D>
struct Args {
  const uint16_t* q;
  int64_t ldq;
  const int32_t* table;
  int64_t ldt;
  const int32_t* lens;
  const int32_t* row_start;
  const int32_t* pos;
  const int32_t* tree;
  const uint16_t* gamma;
  uint16_t* out;
  int64_t ldo;
  float* lse;
  int32_t* count;   // [kMaxBlocks], zero between calls
  float2* ml;       // [2 kMaxBlocks][rows of a unit]: maximum and sum (base 2)
  float* acc;       // [2 kMaxBlocks][rows of a unit][D]
  int32_t* dev_status;
  tfd_kv_pages c;
  int rows, q_heads, group, max_pages, requests, max_new, window, qk;
  float eps, scale;  // scale: times log2 e
  RopeTurns<D> turns;
};

// Tokens of a slice and of a tile; bytes of a vector; stage of a warp: keys, values, scales, which tokens are there.
template <int D, bool kF8>
struct Shape {
  static constexpr int kRow = D * (kF8 ? 1 : 2);
  static constexpr int kKeys = kRow == 256 ? 16 : 32;
  static constexpr int kTile = kW * kKeys;
  static constexpr int kPlane = kKeys * kRow;
  static constexpr int kScales = 2 * kPlane;               // offset: kKeys floats of k, then of v
  static constexpr int kMask = kScales + (kF8 ? 8 * kKeys : 0);
  static constexpr int kStage = kMask + 16;
  static constexpr int kRing = (kW * kStages * kStage + 127) / 128 * 128;
};

__device__ __forceinline__ uint32_t sa(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
template <bool kHalf>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kHalf)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 2^x (2^-22 relative); 0 for -inf.
__device__ __forceinline__ float exp2_(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 codes (the low half of w) as f16.
__device__ __forceinline__ uint32_t e4m3_f16x2(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}
// Two E4M3 codes, each in the high byte of a half word, as bf16: the code's 7 bits placed 4 lower read
// as its value times 2^-120 (exact, as are all E4M3 values; a NaN code reads as 480).
__device__ __forceinline__ uint32_t e4m3_bf16x2(uint32_t w) {
  const uint32_t x = (w & 0x80008000u) | ((w >> 4) & 0x07F007F0u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x7B807B80u));  // 2^120
  return r;
}
__device__ __forceinline__ bool finite_(float x) { return fabsf(x) < INFINITY; }

// Where 16-byte piece c of row r of a plane stands.
template <int kRow>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  if (kRow == 64) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return (uint32_t)(r * kRow + ((c ^ (r & 7)) << 4));
}

struct Request {
  int r, row0, n, len;   // its rows and the tokens before them
  int64_t base;          // first tile of its first unit on the line
  int tile0, tiles, mt;  // first tile of its tokens that a row can see, tiles from there, units a head
  bool bad;
};

// Request r's part of the line.
template <int D, bool kF8, int MT>
__device__ __forceinline__ Request request(const Args<D>& a, int r) {
  using S = Shape<D, kF8>;
  Request q;
  q.r = r;
  q.row0 = a.row_start[r];
  const int64_t n = (int64_t)a.row_start[r + 1] - q.row0;
  q.len = a.lens[r];
  q.base = 0;
  q.bad = q.row0 < 0 || n < 0 || n > a.max_new || q.row0 + n > a.rows || q.len < 0 ||
          (n > 0 && (q.len + n > (int64_t)a.max_pages * a.c.page_size || q.len + n > kMostTokens));
  q.n = q.bad ? 0 : (int)n;
  const int64_t lo = a.window >= 0 ? (int64_t)q.len - a.window - (a.tree ? 1 : 0) : 0;
  q.tile0 = q.n > 0 && lo > 0 ? (int)(lo / S::kTile) : 0;
  q.tiles = q.n > 0 ? (q.len + q.n - 1) / S::kTile + 1 - q.tile0 : 0;
  q.mt = (q.n * a.group + 16 * MT - 1) / (16 * MT);
  return q;
}

template <int D, bool kF8, int MT>
struct Smem {
  using S = Shape<D, kF8>;
  static constexpr int kM = 16 * MT;                  // rows of a unit
  static constexpr int kQ = S::kRing;                 // two parts of q', [kM] rows of 2 D bytes each
  static constexpr int kRows = kQ + 2 * kM * 2 * D;   // per row: first cached token seen, new ones seen, factor
  static constexpr int kStat = kQ;                    // [kW][kM] maximum and sum, when q' is done with
  static constexpr int kBytes = kRows + kM * 12;
  static_assert(kW * kM * 8 <= kRows - kQ, "the warps' statistics fit the place of q'");
  static constexpr int kPitch = D + 8;                // floats of a row of the warps' sums, in the ring
  static_assert(kW * kM * kPitch * 4 <= S::kRing, "the warps' sums fit the ring");
  static_assert(kMaxBlocks * kM * 4 <= S::kRing, "the pieces' weights fit the ring");
};

template <int D, bool kF8, int MT>
__global__ void __launch_bounds__(kT, kPerSm) paged_attn_kernel(const __grid_constant__ Args<D> a) {
  using S = Shape<D, kF8>;
  using M = Smem<D, kF8, MT>;
  constexpr int kM = M::kM, kRow = S::kRow, kKeys = S::kKeys, NT = kKeys / 8, E = D / 32;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ int64_t scan[kW];
  __shared__ int64_t s_base;
  __shared__ int s_r, s_last;
  tfd_host::after_previous();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.c.heads, ps = a.c.page_size;

  // ---- this block's stretch of the line -----------------------------------------------------------
  int64_t total;
  {
    const int per = (a.requests + kT - 1) / kT;
    const int r0 = min(a.requests, tid * per), r1 = min(a.requests, r0 + per);
    int64_t mine = 0;
    for (int r = r0; r < r1; ++r) {
      const Request q = request<D, kF8, MT>(a, r);
      if (q.bad && blockIdx.x == 0) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
      mine += (int64_t)q.tiles * q.mt * H;
    }
    int64_t x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t lo = __shfl_up_sync(0xffffffffu, (uint32_t)x, d);
      const uint32_t hi = __shfl_up_sync(0xffffffffu, (uint32_t)((uint64_t)x >> 32), d);
      if (lane >= d) x += (int64_t)((uint64_t)hi << 32 | lo);
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    total = 0;
    int64_t before = x - mine;
    for (int w = 0; w < kW; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    const int64_t share = (total + gridDim.x - 1) / gridDim.x, t0 = blockIdx.x * share;
    if (t0 >= total) return;  // block-uniform
    if (before <= t0 && t0 < before + mine) {  // one thread
      int r = r0;
      for (; r < r1 - 1; ++r) {
        const Request q = request<D, kF8, MT>(a, r);
        const int64_t u = (int64_t)q.tiles * q.mt * H;
        if (t0 < before + u) break;
        before += u;
      }
      s_r = r;
      s_base = before;
    }
    __syncthreads();
  }
  const int64_t share = (total + gridDim.x - 1) / gridDim.x;
  int64_t t = blockIdx.x * share;
  const int64_t t_end = t + share < total ? t + share : total;
  Request rq = request<D, kF8, MT>(a, s_r);
  rq.base = s_base;

  unsigned char* ring = sm + warp * kStages * S::kStage;
  const uint32_t s_ring = sa(ring), s_q = sa(sm + M::kQ);
  int* s_lo = reinterpret_cast<int*>(sm + M::kRows);
  uint32_t* s_new = reinterpret_cast<uint32_t*>(s_lo + kM);
  float* s_fac = reinterpret_cast<float*>(s_new + kM);
  float2* s_stat = reinterpret_cast<float2*>(sm + M::kStat);
  const int qr = lane >> 2, qc = lane & 3;  // this lane's row (and row + 8) and columns of an accumulator

  while (t < t_end) {
    while (t >= rq.base + (int64_t)rq.tiles * rq.mt * H) {
      const int64_t next = rq.base + (int64_t)rq.tiles * rq.mt * H;
      if (rq.r + 1 >= a.requests) return;  // the line ends before: lengths that changed meanwhile
      rq = request<D, kF8, MT>(a, rq.r + 1);
      rq.base = next;
    }
    const int64_t unit = (t - rq.base) / rq.tiles;
    const int first = (int)(t - rq.base - unit * rq.tiles);  // tile of the unit
    const int h = (int)(unit / rq.mt), m0 = (int)(unit - (int64_t)h * rq.mt) * kM;
    const int cnt = (int)min((int64_t)(rq.tiles - first), t_end - t);
    const int valid = min(kM, rq.n * a.group - m0);
    const int tokens = rq.len + rq.n;
    const int32_t* table = a.table + rq.r * a.ldt;
    const unsigned char* kbase = (const unsigned char*)a.c.k;
    const unsigned char* vbase = (const unsigned char*)a.c.v;

    // ---- a warp's slice of a tile on its way ------------------------------------------------------
    int page = 0;  // of this lane's token of the slice that is fetched next
    auto token_of = [&](int i) {
      return (int64_t)(rq.tile0 + first + i) * S::kTile + warp * kKeys + (lane & (kKeys - 1));
    };
    auto look_up = [&](int i) {
      const int64_t tok = token_of(i);
      page = i < cnt && tok < tokens ? table[(uint32_t)tok / (uint32_t)ps] : -1;
    };
    auto fetch = [&](int i) {
      if (i < cnt) {
        const int64_t tok = token_of(i);
        const uint32_t st = s_ring + (uint32_t)(i % kStages) * S::kStage;
        const bool in = page >= 0 && page < a.c.pages;
        if (tok < tokens && !in) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
        const int at = (int)((uint32_t)tok % (uint32_t)ps);
        const int64_t off =
            in ? (page * a.c.page_stride + at * a.c.token_stride + h * a.c.head_stride) * (kF8 ? 1 : 2)
               : -1;
        const uint32_t there = __ballot_sync(0xffffffffu, in);
        if (lane == 0) *reinterpret_cast<uint32_t*>(ring + (i % kStages) * S::kStage + S::kMask) =
              kKeys == 32 ? there : there & 0xffffu;
        constexpr int L = kRow / 16, P = 32 / L;  // lanes of a vector, vectors a step
#pragma unroll
        for (int j = 0; j < kKeys / P; ++j) {
          const int row = j * P + lane / L, c = lane % L;
          const int64_t o = __shfl_sync(0xffffffffu, off, row);
          const uint32_t d = st + piece<kRow>(row, c);
          const int64_t from = o >= 0 ? o + 16 * c : 0;
          copy16(d, kbase + from, o >= 0);
          copy16(d + S::kPlane, vbase + from, o >= 0);
        }
        if (kF8) {
          const int64_t sc = in ? ((int64_t)page * H + h) * ps + at : 0;
          copy4(st + S::kScales + 4 * lane, a.c.k_scales + sc, in);
          copy4(st + S::kScales + 4 * kKeys + 4 * lane, a.c.v_scales + sc, in);
        }
      }
      copy_commit();
      look_up(i + 1);
    };
    look_up(0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    // ---- q' in two parts, and what each row sees ----------------------------------------------------
    {
      int at_row = -1;
      float sn[E], cs[E];
#pragma unroll
      for (int e = 0; e < E; ++e) sn[e] = cs[e] = 0.0f;
      for (int i = warp; i < kM; i += kW) {  // a row a warp
        uint32_t hi[E / 2], lo[E / 2];
        float fac = 1.0f;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) hi[e] = lo[e] = 0u;
        if (i < valid) {
          const int j = (m0 + i) / a.group, hq = h * a.group + (m0 + i) % a.group;
          const int row = rq.row0 + j;
          float x[E];
          const uint16_t* src = a.q + row * a.ldq + (int64_t)hq * D + E * lane;
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(src + e);
            x[e] = bf16_lo(w);
            x[e + 1] = bf16_hi(w);
          }
          const uint32_t rows_there = rq.n == 32 ? 0xffffffffu : (1u << rq.n) - 1u;
          const uint32_t word = a.tree ? (uint32_t)a.tree[row] & rows_there : 0u;
          const int depth = rq.len + (a.tree ? __popc(word) - 1 : j);
          if (a.qk & TFD_QK_NORM) norm_rows<D>(x, a.gamma, a.eps);
          if (a.qk & TFD_QK_ROPE) {
            if (j != at_row) {
              int p = a.pos ? a.pos[row] : depth;
              if (p < 0) {
                if (a.pos && lane == 0) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
                p = 0;
              }
              rope_sincos<D>(p, a.turns, sn, cs);
              at_row = j;
            }
            rotate<D>(x, sn, cs);
          }
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] *= a.scale;
          if (kF8) {  // into f16's range: the largest magnitude in [1, 2)
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(x[e]));
            top = warp_max(top);
            if (top > 0.0f && finite_(top)) {
              int ex = (int)((__float_as_uint(top) >> 23) & 0xffu) - 127;
              ex = max(-126, min(126, ex));
              const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
              fac = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
              for (int e = 0; e < E; ++e) x[e] *= inv;
            }
          }
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            float rest[2];
            hi[e / 2] = kF8 ? f16x2(x[e], x[e + 1]) : bf16x2(x[e], x[e + 1]);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t w = b ? hi[e / 2] >> 16 : hi[e / 2] & 0xffffu;
              const float back = kF8 ? __half2float(__ushort_as_half((uint16_t)w))
                                     : __uint_as_float(w << 16);
              rest[b] = finite_(back) ? x[e + b] - back : 0.0f;
            }
            lo[e / 2] = kF8 ? f16x2(rest[0], rest[1]) : bf16x2(rest[0], rest[1]);
          }
          if (lane == 0) {
            // the new tokens that the row sees, and its first cached one
            uint32_t sees = 0u;
            const int64_t from = a.window >= 0 ? (int64_t)depth - a.window : -1;
            for (int jj = 0; jj < rq.n; ++jj) {
              const int dj =
                  rq.len + (a.tree ? __popc((uint32_t)a.tree[rq.row0 + jj] & rows_there) - 1 : jj);
              const bool on = (a.tree ? (word >> jj) & 1u : jj <= j) && dj >= from;
              sees |= (uint32_t)on << jj;
            }
            s_new[i] = sees;
            s_lo[i] = from > 0 ? (int)min(from, (int64_t)rq.len) : 0;
          }
        } else if (lane == 0) {
          s_new[i] = 0u;
          s_lo[i] = rq.len;
        }
        if (lane == 0) s_fac[i] = fac;
        // element d of a row stands at its place in the k order of the products: as it is for bf16; for
        // E4M3, whose lanes hold 4 codes in a row, 4t + {0, 1} at 2t + {0, 1} and 4t + {2, 3} at 8 + 2t + {0, 1}
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const int d = E * lane + e, in = d & 15;
          const int to = kF8 ? (d & ~15) + (in >> 2) * 2 + ((in & 2) ? 8 : 0) : d;
          const uint32_t at = (uint32_t)M::kQ + piece<2 * D>(i, to >> 3) + (to & 7) * 2;
          *reinterpret_cast<uint32_t*>(sm + at) = hi[e / 2];
          *reinterpret_cast<uint32_t*>(sm + at + kM * 2 * D) = lo[e / 2];
        }
      }
    }
    __syncthreads();
    uint32_t aq[MT == 1 ? D / 16 : 1][2][4];
    const int a_row = lane & 15, a_piece = lane >> 4;  // ldmatrix: rows and halves of an A tile
    if (MT == 1) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int part = 0; part < 2; ++part)
          ldsm4(aq[MT == 1 ? k : 0][part],
                s_q + part * kM * 2 * D + piece<2 * D>(a_row, 2 * k + a_piece));
    }
    float o[MT][D / 8][4], mx[MT][2], sum[MT][2], fac[MT][2];
    int lo[MT][2];
    uint32_t fresh[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][n][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[m][e] = -INFINITY;
        sum[m][e] = 0.0f;
        lo[m][e] = s_lo[16 * m + qr + 8 * e];
        fresh[m][e] = s_new[16 * m + qr + 8 * e];
        fac[m][e] = kF8 ? s_fac[16 * m + qr + 8 * e] : 1.0f;
      }
    }
    int lo_most = 0;  // from here to the last cached token every row sees all
    for (int i = 0; i < valid; ++i) lo_most = max(lo_most, s_lo[i]);

    // ---- the warp's slices --------------------------------------------------------------------------
    for (int i = 0; i < cnt; ++i) {
      copy_wait<kStages - 2>();
      __syncwarp();  // slice i is here for all lanes, and all are done with slice i - 1
      fetch(i + kStages - 1);
      const int key0 = (int)((int64_t)(rq.tile0 + first + i) * S::kTile) + warp * kKeys;
      if (key0 >= tokens) continue;  // warp-uniform
      const uint32_t st = s_ring + (uint32_t)(i % kStages) * S::kStage;
      const unsigned char* stage = ring + (i % kStages) * S::kStage;
      const uint32_t there = *reinterpret_cast<const uint32_t*>(stage + S::kMask);
      constexpr uint32_t kAll = kKeys == 32 ? 0xffffffffu : 0xffffu;

      float s[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[m][n][e] = 0.0f;
      if (kF8) {
#pragma unroll
        for (int k = 0; k < D / 16; k += 2) {
          uint32_t af[2][MT][2][4];
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int part = 0; part < 2; ++part) {
                if (MT == 1) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) af[kk][m][part][e] = aq[MT == 1 ? k + kk : 0][part][e];
                } else {
                  ldsm4(af[kk][m][part], s_q + part * kM * 2 * D +
                                             piece<2 * D>(16 * m + a_row, 2 * (k + kk) + a_piece));
                }
              }
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];  // keys 8n.. at pieces k, k + 1; keys 8n + 8.. at both
            ldsm4(b, st + piece<kRow>(8 * n + (lane & 7) + ((lane >> 4) << 3), k + ((lane >> 3) & 1)));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t b0 = e4m3_f16x2((uint16_t)b[q]), b1 = e4m3_f16x2((uint16_t)(b[q] >> 16));
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                mma<true>(s[m][n + (q >> 1)], af[q & 1][m][0], b0, b1);
                mma<true>(s[m][n + (q >> 1)], af[q & 1][m][1], b0, b1);
              }
            }
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t af[MT][2][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              if (MT == 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) af[m][part][e] = aq[MT == 1 ? k : 0][part][e];
              } else {
                ldsm4(af[m][part],
                      s_q + part * kM * 2 * D + piece<2 * D>(16 * m + a_row, 2 * k + a_piece));
              }
            }
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            ldsm4(b, st + piece<kRow>(8 * n + (lane & 7) + ((lane >> 4) << 3),
                                      2 * k + ((lane >> 3) & 1)));
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int part = 0; part < 2; ++part) {
                mma<false>(s[m][n], af[m][part], b[0], b[1]);
                mma<false>(s[m][n + 1], af[m][part], b[2], b[3]);
              }
          }
        }
      }
      const float* ks = reinterpret_cast<const float*>(stage + S::kScales);
      if (kF8) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 f = *reinterpret_cast<const float2*>(ks + 8 * n + 2 * qc);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            s[m][n][0] *= fac[m][0] * f.x;
            s[m][n][1] *= fac[m][0] * f.y;
            s[m][n][2] *= fac[m][1] * f.x;
            s[m][n][3] *= fac[m][1] * f.y;
          }
        }
      }
      // hidden tokens
      const bool hidden = there != kAll || key0 + kKeys > rq.len || key0 < lo_most;  // warp-uniform
      if (hidden) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = 8 * n + 2 * qc + (e & 1), key = key0 + c, j = key - rq.len;
            const bool is = (there >> c) & 1u;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const bool on = is && (j < 0 ? key >= lo[m][e >> 1]
                                           : j < 32 && ((fresh[m][e >> 1] >> (j & 31)) & 1u));
              if (!on) s[m][n][e] = -INFINITY;
            }
          }
      }
      // running maximum
      float base[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(s[m][0][2 * e], s[m][0][2 * e + 1]);
#pragma unroll
          for (int n = 1; n < NT; ++n) x = fmaxf(x, fmaxf(s[m][n][2 * e], s[m][n][2 * e + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          const float was = mx[m][e];
          x = fmaxf(x, was);
          mx[m][e] = x;
          base[m][e] = x == -INFINITY ? 0.0f : x;
          if (__any_sync(0xffffffffu, x > was)) {
            const float f = exp2_(was - base[m][e]);
            sum[m][e] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[m][n][2 * e] *= f;
              o[m][n][2 * e + 1] *= f;
            }
          }
        }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[m][n][e] = exp2_(s[m][n][e] - base[m][e >> 1]);
            sum[m][e >> 1] += s[m][n][e];
          }
      if (kF8) {  // the values' scales go into the weights; a weight of zero stays zero
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 f = *reinterpret_cast<const float2*>(ks + kKeys + 8 * n + 2 * qc);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[m][n][e] = hidden && s[m][n][e] == 0.0f ? 0.0f : s[m][n][e] * (e & 1 ? f.y : f.x);
        }
      }
      bool odd = false;  // values that are not finite, where a row does not see them all
      if (!kF8 && hidden) {
#pragma unroll 4
        for (int j = lane; j < S::kPlane / 16; j += 32) {
          const uint4 v = *reinterpret_cast<const uint4*>(stage + S::kPlane + 16 * j);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            odd |= (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
        }
        odd = __any_sync(0xffffffffu, odd);
      }
      const uint32_t sv = st + S::kPlane;
      if (kF8 || !odd) {
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k) {
          uint32_t p[MT][2][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float x = s[m][2 * k + b][2 * e], y = s[m][2 * k + b][2 * e + 1];
                const uint32_t w = bf16x2(x, y);
                p[m][0][2 * b + e] = w;
                p[m][1][2 * b + e] = bf16x2(x - bf16_lo(w), y - bf16_hi(w));
              }
          if (kF8) {
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
              uint32_t v[4];  // codes of dims 32 n + 2 g, + 1 (then 16 more) of tokens 2t, 2t + 1 (then 8 more)
              ldsm4t(v, sv + piece<kRow>(16 * k + (lane & 7) + (((lane >> 3) & 1) << 3),
                                         2 * n + (lane >> 4)));
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint32_t even0 = e4m3_bf16x2(__byte_perm(v[2 * q], 0, 0x2404));
                const uint32_t even1 = e4m3_bf16x2(__byte_perm(v[2 * q + 1], 0, 0x2404));
                const uint32_t odd0 = e4m3_bf16x2(__byte_perm(v[2 * q], 0, 0x3414));
                const uint32_t odd1 = e4m3_bf16x2(__byte_perm(v[2 * q + 1], 0, 0x3414));
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                  for (int part = 0; part < 2; ++part) {
                    mma<false>(o[m][4 * n + 2 * q], p[m][part], even0, even1);
                    mma<false>(o[m][4 * n + 2 * q + 1], p[m][part], odd0, odd1);
                  }
              }
            }
          } else {
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              uint32_t v[4];
              ldsm4t(v, sv + piece<kRow>(16 * k + (lane & 7) + (((lane >> 3) & 1) << 3),
                                         2 * n + (lane >> 4)));
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                  mma<false>(o[m][2 * n], p[m][part], v[0], v[1]);
                  mma<false>(o[m][2 * n + 1], p[m][part], v[2], v[3]);
                }
            }
          }
        }
      } else {
        for (int c = 0; c < kKeys; ++c) {
          const int src = (lane & ~3) | ((c & 7) >> 1);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = 0.0f;
#pragma unroll
              for (int n = 0; n < NT; ++n)
                if (n == c >> 3) x = c & 1 ? s[m][n][2 * e + 1] : s[m][n][2 * e];
              w[e] = __shfl_sync(0xffffffffu, x, src);
            }
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int byte = 2 * (8 * n + 2 * qc + e);
                const float v = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(
                    stage + S::kPlane + piece<kRow>(c, byte >> 4) + (byte & 15)));
                if (w[0] != 0.0f) o[m][n][e] = fmaf(w[0], v, o[m][n][e]);
                if (w[1] != 0.0f) o[m][n][2 + e] = fmaf(w[1], v, o[m][n][2 + e]);
              }
          }
        }
      }
    }

    // ---- the warps' sums added up -------------------------------------------------------------------
    copy_wait<0>();
    __syncthreads();  // the ring is free
    float* sums = reinterpret_cast<float*>(sm);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = sum[m][e];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        const int row = 16 * m + qr + 8 * e;
        if (qc == 0) s_stat[warp * kM + row] = make_float2(mx[m][e], x);
        float* to = sums + (warp * kM + row) * M::kPitch;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          if (kF8) {
            const int d = 16 * (n >> 1) + 4 * qc + (n & 1);
            to[d] = o[m][n][2 * e];
            to[d + 2] = o[m][n][2 * e + 1];
          } else {
            *reinterpret_cast<float2*>(to + 8 * n + 2 * qc) =
                make_float2(o[m][n][2 * e], o[m][n][2 * e + 1]);
          }
        }
      }
    __syncthreads();
    const bool whole = cnt == rq.tiles;
    const int64_t line0 = rq.base + unit * rq.tiles;     // the unit's first tile on the line
    const int b0 = (int)(line0 / share), pieces = (int)((line0 + rq.tiles - 1) / share) - b0 + 1;
    const int slot = 2 * blockIdx.x + (first == 0 ? 1 : 0);
    auto put_row = [&](int i, int d, const float4& v, float mxi, float l) {
      const int row = rq.row0 + (m0 + i) / a.group, hq = h * a.group + (m0 + i) % a.group;
      const float inv = l > 0.0f ? 1.0f / l : l == l ? 0.0f : l;
      uint2 w;
      w.x = bf16x2(v.x * inv, v.y * inv);
      w.y = bf16x2(v.z * inv, v.w * inv);
      if (l == 0.0f) w = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(a.out + row * a.ldo + (int64_t)hq * D + d) = w;
      if (a.lse && d == 0)
        a.lse[(int64_t)row * a.q_heads + hq] =
            l == 0.0f ? -INFINITY : (mxi + log2f(l)) * 0.6931471805599453f;
    };
    for (int i = tid / (D / 4); i < valid; i += kT / (D / 4)) {
      const int d = tid % (D / 4) * 4;
      float top = -INFINITY, l = 0.0f;
      float2 st[kW];
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        st[w] = s_stat[w * kM + i];
        top = fmaxf(top, st[w].x);
      }
      const float b = top == -INFINITY ? 0.0f : top;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const float f = exp2_(st[w].x - b);
        const float4 x = *reinterpret_cast<const float4*>(sums + (w * kM + i) * M::kPitch + d);
        l += f * st[w].y;
        v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
      }
      if (whole) {
        put_row(i, d, v, top, l);
      } else {
        __stcg(reinterpret_cast<float4*>(a.acc + ((int64_t)slot * kM + i) * D + d), v);
        if (d == 0) __stcg(a.ml + (int64_t)slot * kM + i, make_float2(top, l));
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int was = atomicAdd(a.count + b0, 1);
        s_last = was == pieces - 1;
        if (s_last) a.count[b0] = 0;
      }
      __syncthreads();
      if (s_last) {  // all pieces are there: added in their order
        __threadfence();
        auto slot_of = [&](int p) { return (int64_t)(p == 0 ? 2 * b0 + 1 : 2 * (b0 + p)) * kM; };
        float* weight = reinterpret_cast<float*>(sm);  // [valid][pieces]
        for (int i = warp; i < valid; i += kW) {
          float top = -INFINITY, l = 0.0f;
          for (int p = lane; p < pieces; p += 32) top = fmaxf(top, __ldcg(a.ml + slot_of(p) + i).x);
          top = warp_max(top);
          const float b = top == -INFINITY ? 0.0f : top;
          for (int p = lane; p < pieces; p += 32) {
            const float2 st = __ldcg(a.ml + slot_of(p) + i);
            const float f = exp2_(st.x - b);
            weight[i * pieces + p] = f;
            l += f * st.y;
          }
          l = warp_sum(l);
          if (lane == 0) s_stat[i] = make_float2(top, l);
        }
        __syncthreads();
        for (int i = tid / (D / 4); i < valid; i += kT / (D / 4)) {
          const int d = tid % (D / 4) * 4;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
          for (int p = 0; p < pieces; ++p) {
            const float f = weight[i * pieces + p];
            const float4 x = __ldcg(reinterpret_cast<const float4*>(a.acc + (slot_of(p) + i) * D + d));
            v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
          }
          const float2 st = s_stat[i];
          put_row(i, d, v, st.x, st.y);
        }
      }
    }
    __syncthreads();  // shared memory is free for the next piece
    t += cnt;
  }
}

// Rows of a unit: 16 where no request can have more, else 32.
inline int unit_rows(int max_new, int group) { return max_new * group <= 16 ? 16 : 32; }

inline size_t workspace(int max_new, int group, int dim) {
  const size_t rows = (size_t)2 * kMaxBlocks * unit_rows(max_new, group);
  return kMaxBlocks * 4 + rows * 8 + rows * dim * 4;
}

template <int D, bool kF8, int MT>
tfd_status launch(const Args<D>& a, cudaStream_t stream) {
  int dev = 0;
  const int sms = tfd_host::device_sms(dev);
  const int blocks = std::min(kMaxBlocks, std::max(1, sms * kPerSm));
  constexpr int smem = Smem<D, kF8, MT>::kBytes;
  return tfd_host::launch_clusters<paged_attn_kernel<D, kF8, MT>>(a, dev, blocks, 1, kT, smem, smem,
                                                                  stream);
}

template <int D>
tfd_status launch_dim(Args<D>& a, float rope_base, cudaStream_t stream) {
  if (a.qk & TFD_QK_ROPE) a.turns = tfd_host::rope_turns<D>(rope_base);
  const bool one = unit_rows(a.max_new, a.group) == 16;
  if (a.c.fmt == TFD_KV_E4M3)
    return one ? launch<D, true, 1>(a, stream) : launch<D, true, 2>(a, stream);
  return one ? launch<D, false, 1>(a, stream) : launch<D, false, 2>(a, stream);
}

}  // namespace

extern "C" size_t tfd_paged_attn_workspace(int max_new, int q_heads, int heads, int dim) {
  if (max_new < 1 || max_new > TFD_MAX_ROWS || heads < 1 || heads > 1024 || q_heads < heads ||
      q_heads % heads || q_heads / heads > 64 || (dim != 64 && dim != 128))
    return 0;
  return workspace(max_new, q_heads / heads, dim);
}

extern "C" tfd_status tfd_paged_attn(const void* q, int64_t ldq, int rows, int q_heads,
                                     const tfd_kv_pages* cache, const int32_t* table, int64_t ldt,
                                     int max_pages, const int32_t* lens, const int32_t* row_start,
                                     int requests, int max_new, const int32_t* pos,
                                     const int32_t* tree, int window, int qk, const void* q_gamma,
                                     float eps, float rope_base, float scale, void* out, int64_t ldo,
                                     float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                                     void* stream) {
  using tfd_host::aligned;
  if (!q || !table || !lens || !row_start || !out) return TFD_ERR_INVALID;
  const tfd_status st = tfd_paged::check_cache(cache);
  if (st != TFD_OK) return st;
  const tfd_kv_pages& c = *cache;
  if (rows < 1 || requests < 1 || max_new < 1 || max_new > TFD_MAX_ROWS || max_pages < 1 ||
      ldt < max_pages || window < -1)
    return TFD_ERR_INVALID;
  if (q_heads < c.heads || q_heads % c.heads || q_heads / c.heads > 64) return TFD_ERR_INVALID;
  if (!tfd_paged::check_qk(qk, eps, rope_base) || !(scale >= 0.0f) || !(scale <= 3.0e38f))
    return TFD_ERR_INVALID;
  const int64_t width = (int64_t)q_heads * c.dim;
  if (ldq < width || ldq % 8 || ldo < width || ldo % 8) return TFD_ERR_INVALID;
  if (requests > TFD_MAX_REQUESTS || ldq > ((int64_t)1 << 30) || ldo > ((int64_t)1 << 30) ||
      ldt > ((int64_t)1 << 40) || (int64_t)rows * q_heads > 2147483647)
    return TFD_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(row_start, 4) || !aligned(pos, 4) || !aligned(tree, 4) || !aligned(q_gamma, 2) ||
      !aligned(lse, 4) || !aligned(dev_status, 4) || !aligned(ws, 16))
    return TFD_ERR_INVALID;
  const int group = q_heads / c.heads;
  const size_t need = workspace(max_new, group, c.dim);
  if (!ws || ws_bytes < need) return TFD_ERR_WORKSPACE;
  const struct {
    const void* p;
    int64_t bytes;
  } in[] = {{q, ((int64_t)(rows - 1) * ldq + width) * 2},
            {table, ((int64_t)(requests - 1) * ldt + max_pages) * 4},
            {lens, requests * 4ll},
            {row_start, requests * 4ll + 4},
            {pos, rows * 4ll},
            {tree, rows * 4ll},
            {q_gamma, c.dim * 2}},
    outs[] = {{out, ((int64_t)(rows - 1) * ldo + width) * 2},
              {lse, (int64_t)rows * q_heads * 4},
              {ws, (int64_t)need},
              {dev_status, 4}};
  for (int i = 0; i < 4; ++i) {
    for (const auto& x : in)
      if (tfd_host::overlap(outs[i].p, outs[i].bytes, x.p, x.bytes)) return TFD_ERR_INVALID;
    for (int j = i + 1; j < 4; ++j)
      if (tfd_host::overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes))
        return TFD_ERR_INVALID;
    if (outs[i].p && tfd_paged::overlaps_cache(c, outs[i].p, outs[i].bytes)) return TFD_ERR_INVALID;
  }
  const float sc =
      (float)((scale > 0.0f ? (double)scale : 1.0 / std::sqrt((double)c.dim)) * 1.4426950408889634);
  char* w = (char*)ws;
  const size_t slots = (size_t)2 * kMaxBlocks * unit_rows(max_new, group);
  int32_t* count = (int32_t*)w;
  float2* ml = (float2*)(w + kMaxBlocks * 4);
  float* acc = (float*)(w + kMaxBlocks * 4 + slots * 8);
  cudaStream_t s = tfd_host::as_stream(stream);
#define TFD_ATTN_DIM(D)                                                                          \
  if (c.dim == D) {                                                                              \
    Args<D> a = {(const uint16_t*)q, ldq, table, ldt, lens, row_start, pos, tree,                \
                 (const uint16_t*)q_gamma, (uint16_t*)out, ldo, lse, count, ml, acc, dev_status, \
                 c, rows, q_heads, group, max_pages, requests, max_new, window, qk, eps, sc, {}}; \
    return launch_dim<D>(a, rope_base, s);                                                       \
  }
  TFD_ATTN_DIM(64)
  TFD_ATTN_DIM(128)
#undef TFD_ATTN_DIM
  return TFD_ERR_UNSUPPORTED;
}
