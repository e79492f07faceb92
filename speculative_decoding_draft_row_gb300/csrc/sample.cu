// sample.cu - draws one token a row from its logits and a given random number, after temperature,
// top-k, top-p and min-p, optionally with the whole filtered distribution.
//
// Weights are exact integers (weight.cuh), so a row's sums are the same in any order. One
// thread-block cluster takes a row, each block a contiguous part of its columns (kept in shared
// memory where they fit), each warp a contiguous part of the block's. After the row's largest logit
// (one cluster barrier) a row goes one of three ways:
//  A. no top-k, no top-p: every warp sums its weights (those that min_p keeps); one barrier.
//  B. top-k up to the list's length: the k-th largest of the threads' own maxima bounds the k-th
//     largest logit from below (k threads each hold a logit at least that large). A histogram of
//     the maxima over log2 of the weight finds a bin edge under it, and only the threads whose
//     maximum reaches the edge look through their columns again; little more than k columns go to
//     every block's list, and each block resolves top-k and top-p on the list alone.
//  C. top-p alone (or what B cannot hold): the histogram takes every column's weight, as three
//     integer pieces that shared-memory adds without a carry; the bin in which the border falls is
//     found, its columns go to the lists, and each block resolves the border on its list. A bin
//     with more columns than the list is split again by the columns' 64-bit (value, id) keys until
//     it fits (equal logits differ by their ids, so this ends).
// The blocks' kept masses then name the block that holds the drawn column, which finds the warp,
// which scans its columns. The histogram is summed across the cluster through distributed shared
// memory, a share of the bins by each block, into every block, so each finds the border's bin for
// itself; the lists and, behind way C, the shares of that block's masses cost a barrier more each.
//
// Bound by the barriers and the block's work between them where rows are few (1 x 4096 with all
// filters 10.9 us, 4 x 163840 with top-p and distributions 30.2, 16 x 163840 bf16 with mixed filters
// 37.4), by the weights' instructions where they are many (33 x 50021 without filters 14.3 us, 96 x
// 163840 with mixed filters and distributions 133, of 19 for the bytes).
#include <cooperative_groups.h>

#include "launch.cuh"
#include "weight.cuh"

namespace {

using namespace tfd;
namespace cg = cooperative_groups;

constexpr int kT = 512;
constexpr int kW = kT / 32;
constexpr int kBins = 1024;
constexpr int kPer = kBins / kT;
constexpr int kList = 1024;      // columns of a list
constexpr int kRank = 128;       // lists up to here are ranked outright (256: up to 10 us more)
constexpr int kMaxC = tfd_host::kMaxCluster;
constexpr int kMaxPart = 65536;  // columns of a block, or a few more: 15-bit pieces sum within 32 bits

struct Args {
  const void* logits;
  int64_t n, ld;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  const int32_t* id_map;
  int32_t* ids;
  float* prob;
  int64_t ldt;
  float* probs;
  int64_t ldp;
  int32_t* dev_status;
};

// A sum of weights in three pieces (bits 0-14, 15-29, 30-43), for adds without carries.
struct Pieces {
  uint32_t lo[kBins], mid[kBins], top[kBins];
};

struct Shared {
  unsigned long long tab[128];
  uint32_t cnt[kBins];  // this block's histogram: columns, and their weights
  Pieces w;
  uint32_t rcnt[kBins];  // the row's
  uint64_t rmass[kBins];
  uint64_t lent[kList];           // the list, in every block: logit bits, column
  uint64_t lkey[kList], lw[kList];  // its keys (own columns on their way out before that), weights
  uint16_t lmem[kList];           // entries of the list's border bin
  uint32_t ltotal[2];             // columns sent to this block's list
  float4 cext[kMaxC];             // every block's largest and smallest logit, smallest thread maximum
  uint64_t cdef[2][kMaxC];        // every block's mass above the border bin
  uint64_t ctail[kMaxC];          // and below the histogram
  uint64_t klo[kMaxC], khi[kMaxC];
  uint64_t wsum[kW];              // this block's warps
  uint64_t part[kMaxC][kW];       // and the other blocks' shares of their sums
  uint64_t w64[kW], x64[kW];
  uint32_t w32[kW];
  float wext[3][kW];
  uint32_t cw3[3][kMaxC], ww3[3][kW];  // kept list columns' masses by block and by warp, in pieces
  uint64_t f_above_m, f_in_m, tkey, zk;
  uint32_t f_bin, f_above_n, f_in_n, n_out, base, n_mem;
};

// The border of a filter: columns in bins below `bin` (higher weights) are kept for certain, and of
// `bin` itself those with a key above khi; keys in [klo, khi] are undecided.
struct Border {
  int bin;
  uint64_t klo, khi;
  uint32_t n_above, n_in;
  uint64_t m_above;
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, (unsigned long long)v, m);
  return v;
}

template <bool BF16, bool KEEP>
struct Sampler {
  static constexpr int VE = BF16 ? 8 : 4;  // logits in 16 bytes
  const Args& a;
  Shared& sh;
  uint4* keep;  // this block's logits, where they fit
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int C, rank, row, off, n, nvc, nvw, vcta, vbeg, vend, nvrow;
  const char* base;
  float m, binscale, lfloor;  // largest logit; bins per unit of log2; no logit below has a say
  float log2_minp;
  bool inf;                   // the largest logit is +inf
  Scale sc;
  uint64_t minw;

  __device__ Sampler(const Args& args, Shared& s, uint4* kp) : a(args), sh(s), keep(kp) {
    C = (int)cl.num_blocks();
    rank = (int)cl.block_rank();
    row = blockIdx.x / C;
    n = (int)a.n;
    inf = false;
    const int es = BF16 ? 2 : 4;
    const char* p = (const char*)a.logits + (int64_t)row * a.ld * es;
    off = (int)((uintptr_t)p & 15) / es;
    base = p - off * es;
    const int nv = (off + n + VE - 1) / VE;
    nvrow = nv;
    nvc = (nv + C - 1) / C;
    nvw = (nvc + kW - 1) / kW;
    vcta = rank * nvc;
    vbeg = vcta + warp * nvw;
    vend = min(min(vbeg + nvw, vcta + nvc), nv);
  }

  // 16 bytes of logits; NaN (no weight) where the row does not reach
  __device__ __forceinline__ uint4 load(int v) const {
    const int lo = v * VE - off;
    if (lo >= 0 && lo + VE <= n) return __ldg((const uint4*)base + v);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (BF16) {
        const uint16_t* q = (const uint16_t*)base + (int64_t)v * 8 + 2 * j;
        const int c = lo + 2 * j;
        const uint32_t x = (c >= 0 && c < n) ? q[0] : 0x7FC0u;
        const uint32_t y = (c + 1 >= 0 && c + 1 < n) ? q[1] : 0x7FC0u;
        w[j] = x | (y << 16);
      } else {
        const int c = lo + j;
        w[j] = (c >= 0 && c < n) ? ((const uint32_t*)base)[(int64_t)v * 4 + j] : 0x7FC00000u;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 get(int v) const {
    if (KEEP) return keep[v - vcta];
    const uint4 r = load(v);
    return inf ? only_inf(r) : r;
  }
  // +inf -> 0, all else -> NaN: where the largest logit is +inf, the +inf columns share the mass
  __device__ static uint4 only_inf(const uint4& r) {
    uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = BF16 ? (((w[j] & 0xFFFFu) == 0x7F80u ? 0u : 0x7FC0u) |
                     ((w[j] >> 16) == 0x7F80u ? 0u : 0x7FC00000u))
                  : (w[j] == 0x7F800000u ? 0u : 0x7FC00000u);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ static float elem(const uint4& r, int j) {
    if (BF16) {
      const uint32_t w = (j >> 1) == 0 ? r.x : (j >> 1) == 1 ? r.y : (j >> 1) == 2 ? r.z : r.w;
      return (j & 1) ? bf16_hi(w) : bf16_lo(w);
    }
    return __uint_as_float(j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w);
  }
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int v = vbeg + lane; v < vend; v += 32) {
      const uint4 r = get(v);
#pragma unroll
      for (int j = 0; j < VE; ++j) f(v * VE + j - off, elem(r, j));
    }
  }
  // f(column, logit) for the columns whose logit is in [lo, hi]
  template <class F>
  __device__ __forceinline__ void each_in(float lo, float hi, F f) const {
    for (int v = vbeg + lane; v < vend; v += 32) {
      const uint4 r = get(v);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float l = elem(r, j);
        if (l >= lo && l <= hi) f(v * VE + j - off, l);
      }
    }
  }

  __device__ __forceinline__ float lead(float l) const { return lead_log2(l, m, sc); }
  __device__ __forceinline__ float place(float ph) const { return -ph * binscale; }
  __device__ __forceinline__ int bin_of(float ph) const {
    return min(kBins - 1, (int)place(ph));
  }
  // A logit whose lead_log2 is about ph, less (or more) than its rounding can make.
  __device__ __forceinline__ float logit_at(float ph, bool below) const {
    const float d = ph / sc.hi, slack = (fabsf(m) + fabsf(d)) * 1e-6f;
    if (!(d > -3e38f)) return below ? -INFINITY : m;
    return below ? m + d - slack : m + d + slack;
  }
  __device__ __forceinline__ uint64_t weight(float l) const {
    return weight_of(l, m, sc, sh.tab);
  }
  __device__ __forceinline__ uint64_t key_of(float l, int col) const {
    return make_key(l, a.id_map ? a.id_map[col] : col);
  }

  // The row's largest logit, smallest finite one, and smallest thread maximum; each thread's own.
  __device__ void extremes(float& mn, float& mt, float& own) {
    float mx = -INFINITY;
    mn = mt = INFINITY;
    for (int v0 = vbeg + lane; v0 < vend; v0 += 128) {
      uint4 r[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (v0 + 32 * q < vend) r[q] = load(v0 + 32 * q);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (v0 + 32 * q < vend) {
          if (KEEP) keep[v0 + 32 * q - vcta] = r[q];
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const float x = elem(r[q], j);
            mx = fmaxf(mx, x);  // fmaxf and fminf pass NaN over
            mn = fminf(mn, x == -INFINITY ? INFINITY : x);
          }
        }
    }
    own = mx;
    if (mx > -INFINITY) mt = mx;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mt = fminf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    }
    if (lane == 0) {
      sh.wext[0][warp] = mx;
      sh.wext[1][warp] = mn;
      sh.wext[2][warp] = mt;
    }
    __syncthreads();
    cl.barrier_wait();  // every block runs and has cleared its counters
    if (warp == 0) {
      const int w = lane & (kW - 1);
      mx = sh.wext[0][w];
      mn = sh.wext[1][w];
      mt = sh.wext[2][w];
#pragma unroll
      for (int o = kW / 2; o > 0; o >>= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mt = fminf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      }
      if (lane < C) *cl.map_shared_rank(&sh.cext[rank], lane) = make_float4(mx, mn, mt, 0.0f);
    }
    cl.sync();
    float4 e = sh.cext[0];
    for (int c = 1; c < C; ++c) {
      const float4 x = sh.cext[c];
      e.x = fmaxf(e.x, x.x);
      e.y = fminf(e.y, x.y);
      e.z = fminf(e.z, x.z);
    }
    m = e.x;
    mn = e.y;
    mt = e.z;
  }

  // ---- histogram ----------------------------------------------------------------------------
  __device__ __forceinline__ void pieces_add(uint32_t* lo, uint32_t* mid, uint32_t* top,
                                             uint64_t w) {
    atomicAdd(lo, (uint32_t)w & 0x7FFFu);
    atomicAdd(mid, ((uint32_t)w >> 15) & 0x7FFFu);
    const uint32_t t = (uint32_t)(w >> 30);
    if (t) atomicAdd(top, t);
  }
  __device__ __forceinline__ static uint64_t pieces(uint32_t lo, uint32_t mid, uint32_t top) {
    return lo + ((uint64_t)mid << 15) + ((uint64_t)top << 30);
  }
  __device__ __forceinline__ void mass_add(int b, uint64_t w) {
    pieces_add(&sh.w.lo[b], &sh.w.mid[b], &sh.w.top[b], w);
  }
  __device__ __forceinline__ uint64_t own_mass(int b) const {
    return pieces(sh.w.lo[b], sh.w.mid[b], sh.w.top[b]);
  }
  __device__ void hist_zero() {  // the caller synchronises
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid + i * kT;
      sh.cnt[b] = sh.w.lo[b] = sh.w.mid[b] = sh.w.top[b] = 0u;
    }
  }
  // The blocks' histograms summed into every block's rcnt, rmass: a share of the bins by each.
  __device__ void hist_sum(bool count, bool mass) {
    cl.sync();
    const int per = (kBins + C - 1) / C;
    int g = 1;
    while (4 * g <= C) g *= 2;
    const int sub = tid & (g - 1);
#pragma unroll 1
    for (int i0 = 0; i0 < per; i0 += kT / g) {
      const int i = i0 + tid / g, b = min(rank * per + i, kBins - 1);
      uint32_t c = 0;
      uint64_t w = 0;
      for (int r = sub; r < C; r += g) {
        const Shared* p = cl.map_shared_rank(&sh, r);
        if (count) c += p->cnt[b];
        if (mass) w += pieces(p->w.lo[b], p->w.mid[b], p->w.top[b]);
      }
      for (int o = 1; o < g; o <<= 1) {
        if (count) c += __shfl_xor_sync(0xffffffffu, c, o);
        if (mass) w += __shfl_xor_sync(0xffffffffu, (unsigned long long)w, o);
      }
      if (i < per)
        for (int r = sub; r < C; r += g) {
          Shared* p = cl.map_shared_rank(&sh, r);
          if (count) p->rcnt[b] = c;
          if (mass) p->rmass[b] = w;
        }
    }
    cl.sync();
  }
  // The row's histogram, of the columns down to `cut` (log2 of the weight). Returns the mass of those
  // below, summed over the row: they are many, and no bin of theirs is wanted where the border lies
  // above them.
  __device__ uint64_t hist_row(bool count, bool mass, float cut) {
    uint64_t tail = 0;
    for (int v = vbeg + lane; v < vend; v += 32) {
      const uint4 r = get(v);
#pragma unroll
      for (int j0 = 0; j0 < VE; j0 += 4) {
        uint64_t w[4];
        if (mass) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = weight(elem(r, j0 + j));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float ph = lead(elem(r, j0 + j));
          if (ph >= cut) {
            const int b = bin_of(ph);
            if (count) atomicAdd(&sh.cnt[b], 1u);
            if (mass) mass_add(b, w[j]);
          } else if (mass) {
            tail += w[j];
          }
        }
      }
    }
    if (mass) {
      tail = block_sum(tail);
      if (tid < C) *cl.map_shared_rank(&sh.ctail[rank], tid) = tail;
    }
    hist_sum(count, mass);
    tail = 0;
    if (mass)
      for (int c = 0; c < C; ++c) tail += sh.ctail[c];
    return tail;
  }

  // The first bin at which the running count (or mass) from bin 0 on, n0 and m0 before it, reaches
  // the target; kBins if none does.
  __device__ int find(uint64_t target, bool by_mass, uint32_t n0, uint64_t m0) {
    uint32_t cn[kPer], c = 0;
    uint64_t wn[kPer], w = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c += cn[i] = sh.rcnt[tid * kPer + i];
      w += wn[i] = sh.rmass[tid * kPer + i];
    }
    uint32_t ci = c;
    uint64_t wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, ci, o);
      const uint64_t y = __shfl_up_sync(0xffffffffu, (unsigned long long)wi, o);
      if (lane >= o) {
        ci += x;
        wi += y;
      }
    }
    if (tid == 0) sh.f_bin = kBins;
    if (lane == 31) {
      sh.w32[warp] = ci;
      sh.w64[warp] = wi;
    }
    __syncthreads();
    uint32_t cb = n0 + ci - c;
    uint64_t wb = m0 + wi - w;
    for (int q = 0; q < warp; ++q) {
      cb += sh.w32[q];
      wb += sh.w64[q];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint64_t before = by_mass ? wb : cb, after = by_mass ? wb + wn[i] : cb + cn[i];
      if (before < target && after >= target) {
        sh.f_bin = tid * kPer + i;
        sh.f_above_n = cb;
        sh.f_above_m = wb;
        sh.f_in_n = cn[i];
        sh.f_in_m = wn[i];
      }
      cb += cn[i];
      wb += wn[i];
    }
    __syncthreads();
    return (int)sh.f_bin;
  }
  __device__ void zero_counts() {  // rcnt or rmass where the histogram did not have them
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) sh.rcnt[tid + i * kT] = 0u;
    __syncthreads();
  }
  __device__ void zero_masses() {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) sh.rmass[tid + i * kT] = 0u;
    __syncthreads();
  }

  // ---- the list -----------------------------------------------------------------------------
  // Own columns for the list collect in lkey; n_out counts them.
  __device__ __forceinline__ void list_add(int col, float l) {
    const uint32_t slot = atomicAdd(&sh.n_out, 1u);
    if (slot < (uint32_t)kList)
      sh.lkey[slot] = ((uint64_t)__float_as_uint(l) << 32) | (uint32_t)col;
  }
  // Sends them, and this block's mass above the border, to every block. Returns the columns of the
  // whole row, which are all in the list if they are at most kList. Ends in a cluster barrier.
  __device__ uint32_t list_send(int buf, uint64_t mass) {
    __syncthreads();
    const uint32_t mine = sh.n_out;
    if (tid < C) {
      const uint32_t old = atomicAdd(cl.map_shared_rank(&sh.ltotal[buf], tid), mine);
      if (tid == 0) sh.base = old;  // rank 0's order places the blocks' columns
      *cl.map_shared_rank(&sh.cdef[buf][rank], tid) = mass;
    }
    __syncthreads();
    const uint32_t at = sh.base, cnt = min(mine, (uint32_t)kList);
    for (uint32_t i = tid; i < cnt * C; i += kT) {
      const uint32_t e = i / C, r = i % C;
      if (at + e < (uint32_t)kList) *cl.map_shared_rank(&sh.lent[at + e], r) = sh.lkey[e];
    }
    cl.sync();
    if (tid == 0) sh.n_out = 0;
    return sh.ltotal[buf];
  }
  // Keys and weights of the list.
  __device__ void list_weigh(int cnt) {
    for (int i = tid; i < cnt; i += kT) {
      const uint64_t e = sh.lent[i];
      const float l = __uint_as_float((uint32_t)(e >> 32));
      sh.lkey[i] = key_of(l, (int)(uint32_t)e);
      sh.lw[i] = weight(l);
    }
    __syncthreads();
  }
  // Counts a column of the list in its bin. Equal logits share a bin, and adds to one address go one
  // by one: where the warp has a single bin, one lane adds the sums.
  // `on`: the warp's lanes that have one.
  __device__ __forceinline__ void list_count(unsigned on, int b, uint64_t w) {
    int same;
    __match_all_sync(on, b, &same);
    if (!same) {
      atomicAdd(&sh.cnt[b], 1u);
      mass_add(b, w);
      return;
    }
    const uint32_t lo = __reduce_add_sync(on, (uint32_t)w & 0x7FFFu);
    const uint32_t mid = __reduce_add_sync(on, ((uint32_t)w >> 15) & 0x7FFFu);
    const uint32_t top = __reduce_add_sync(on, (uint32_t)(w >> 30));
    if (lane == __ffs(on) - 1) {
      atomicAdd(&sh.cnt[b], (uint32_t)__popc(on));
      atomicAdd(&sh.w.lo[b], lo);
      atomicAdd(&sh.w.mid[b], mid);
      atomicAdd(&sh.w.top[b], top);
    }
  }
  // The last kept key among the list's columns (n0 columns of mass m0 rank above all of them): the
  // target-th column, or the one at which the running mass reaches the target; and the mass up to
  // and with it. A list too long to rank outright is cut down to one bin of a histogram: first over
  // its places (t0 and mul spread them over the bins), then, for equal logits, over its keys.
  __device__ void list_border(int cnt, float t0, float mul, uint32_t n0, uint64_t m0,
                              uint64_t target, bool by_mass) {
    int mem = cnt;
    uint32_t na = n0;
    uint64_t ma = m0, lo = 0, hi = ~0ull;
    bool split = false;
#pragma unroll 1
    for (int level = 0; mem > kRank && lo < hi; ++level) {
      int shift = 0;
      if (level > 0) {  // the keys left, least and largest
        lo = ~0ull;
        hi = 0;
        for (int j = tid; j < mem; j += kT) {
          const uint64_t k = sh.lkey[sh.lmem[j]];
          lo = min(lo, k);
          hi = max(hi, k);
        }
        block_range(lo, hi);
        shift = max(0, 64 - __clzll((long long)(hi - lo)) - 10);  // (hi - lo) >> shift < 1024
      }
      hist_zero();
      __syncthreads();
      // this thread's entries: their bins, then, with the border bin known, which stay
      int entry[kList / kT], bin[kList / kT], got = 0;
#pragma unroll
      for (int q = 0; q < kList / kT; ++q) {
        const int j = tid + q * kT;
        entry[q] = bin[q] = -1;
        const unsigned on = __ballot_sync(0xffffffffu, j < mem);
        if (j < mem) {
          const int i = split ? sh.lmem[j] : j;
          entry[q] = i;
          if (level > 0) {
            bin[q] = (int)((hi - sh.lkey[i]) >> shift);
          } else {
            const float l = __uint_as_float((uint32_t)(sh.lent[i] >> 32));
            bin[q] = max(0, min(kBins - 1, (int)((place(lead(l)) - t0) * mul)));
          }
          list_count(on, bin[q], sh.lw[i]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int b = tid + i * kT;
        sh.rcnt[b] = sh.cnt[b];
        sh.rmass[b] = own_mass(b);
      }
      if (tid == 0) sh.n_mem = 0;
      __syncthreads();
      const int b = find(target, by_mass, na, ma);
      na = sh.f_above_n;
      ma = sh.f_above_m;
#pragma unroll
      for (int q = 0; q < kList / kT; ++q) got += bin[q] == b;
      uint32_t at = got ? atomicAdd(&sh.n_mem, (uint32_t)got) : 0;
#pragma unroll
      for (int q = 0; q < kList / kT; ++q)
        if (bin[q] == b) sh.lmem[at++] = (uint16_t)entry[q];
      __syncthreads();
      mem = (int)sh.n_mem;
      split = true;
    }
    // 2^g threads rank a column together
    int g = 0;
    while (g < 5 && (mem << (g + 1)) <= kT) ++g;
    const int step = kT >> g, part = tid & ((1 << g) - 1);
    for (int i0 = 0; i0 < mem; i0 += step) {
      const int i = i0 + (tid >> g);
      const int ii = i < mem ? (split ? sh.lmem[i] : i) : 0;
      const uint64_t k = sh.lkey[ii], w = sh.lw[ii];
      const uint32_t col = (uint32_t)sh.lent[ii];
      uint32_t above = 0;
      uint64_t before = 0;
      for (int j = part; j < mem; j += 1 << g) {
        const int jj = split ? sh.lmem[j] : j;
        const uint64_t kj = sh.lkey[jj];
        if (kj > k || (kj == k && (uint32_t)sh.lent[jj] < col)) {
          ++above;
          before += sh.lw[jj];
        }
      }
      for (int o = 1; o < (1 << g); o <<= 1) {
        above += __shfl_xor_sync(0xffffffffu, above, o);
        before += __shfl_xor_sync(0xffffffffu, (unsigned long long)before, o);
      }
      above += na;
      before += ma;
      const bool hit = by_mass ? (before < target && before + w >= target)
                               : (uint64_t)above + 1 == target;
      if (hit && i < mem && part == 0) {
        sh.tkey = k;
        sh.zk = before + w;
      }
    }
    __syncthreads();
  }

  // ---- way C: borders in the row's histogram --------------------------------------------------
  // Splits the border's bin by its columns' keys until the undecided columns fit the list, or have
  // one key. Overwrites the histogram.
  __device__ void refine(Border& b, uint64_t target, bool by_mass) {
    const int bin = b.bin;
    do {
      uint64_t lo = ~0ull, hi = 0;
      each([&](int col, float l) {
        const float ph = lead(l);
        if (alive(ph) && bin_of(ph) == bin) {
          const uint64_t k = key_of(l, col);
          if (k >= b.klo && k <= b.khi) {
            lo = min(lo, k);
            hi = max(hi, k);
          }
        }
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        lo = min(lo, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)lo, o));
        hi = max(hi, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)hi, o));
      }
      __syncthreads();
      if (lane == 0) {
        sh.w64[warp] = lo;
        sh.x64[warp] = hi;
      }
      __syncthreads();
      if (tid < C) {
        for (int w = 0; w < kW; ++w) {
          lo = min(lo, sh.w64[w]);
          hi = max(hi, sh.x64[w]);
        }
        *cl.map_shared_rank(&sh.klo[rank], tid) = lo;
        *cl.map_shared_rank(&sh.khi[rank], tid) = hi;
      }
      hist_zero();
      cl.sync();
      lo = ~0ull;
      hi = 0;
      for (int c = 0; c < C; ++c) {
        lo = min(lo, sh.klo[c]);
        hi = max(hi, sh.khi[c]);
      }
      const uint64_t span = hi - lo;
      const int shift = max(0, 64 - __clzll((long long)span) - 10);  // (span >> shift) < 1024
      each([&](int col, float l) {
        const float ph = lead(l);
        if (alive(ph) && bin_of(ph) == bin) {
          const uint64_t k = key_of(l, col);
          if (k >= lo && k <= hi) {
            const int s = (int)((hi - k) >> shift);
            atomicAdd(&sh.cnt[s], 1u);
            mass_add(s, weight(l));
          }
        }
      });
      hist_sum(true, true);
      const int s = find(target, by_mass, b.n_above, b.m_above);
      b.n_above = sh.f_above_n;
      b.m_above = sh.f_above_m;
      b.n_in = sh.f_in_n;
      b.khi = hi - ((uint64_t)s << shift);
      const uint64_t width = (1ull << shift) - 1;
      b.klo = b.khi - lo < width ? lo : b.khi - width;
      if (b.n_in > (uint32_t)kList && b.klo == b.khi && tid == 0) {  // one key: all of it is kept
        sh.tkey = b.klo;
        sh.zk = b.m_above + sh.f_in_m;
      }
    } while (b.n_in > (uint32_t)kList && b.klo < b.khi);
    __syncthreads();
  }

  // The border at `target` in the row's histogram (which has what it needs), and then in its bin:
  // leaves tkey, zk; returns the columns in the list. cdef[buf] has the blocks' masses above it
  // as far as min_p keeps them.
  __device__ int row_border(int buf, uint64_t target, bool by_mass, bool mass) {
    Border b;
    b.bin = find(target, by_mass, 0, 0);
    b.klo = 0;
    b.khi = ~0ull;
    b.n_above = sh.f_above_n;
    b.m_above = sh.f_above_m;
    // min_p's cut clearly above this bin: it alone decides. Clearly below: it has no say. In between
    // the weights decide, column by column. __log2f is within 2^-21.4 (3.6e-7) absolute near 1, which
    // is many bins where the row spans little (logits 20 apart at a temperature of 1e6: 2.9e-5 in all).
    if (minw) {
      const float at = -log2_minp * binscale, unsure = 1.0f + 4e-7f * binscale;
      if (at < (float)b.bin - unsure) return -1;
      if (at > (float)b.bin + 1.0f + unsure && b.bin < kBins - 1) minw = 0;
    }
    // this block's mass above: from its histogram, or column by column where min_p has a say
    uint64_t sum = 0;
    const bool from_hist = mass && minw == 0;
    if (from_hist)
      for (int i = tid; i < b.bin; i += kT) sum += own_mass(i);
    const float lo = logit_at(-(float)(b.bin + 1) / binscale, true);
    const float hi = from_hist ? logit_at(-(float)b.bin / binscale, false) : INFINITY;
    each_in(b.bin == kBins - 1 ? -INFINITY : lo, hi, [&](int col, float l) {
      const float ph = lead(l);
      if (!alive(ph)) return;
      const int bn = bin_of(ph);
      if (bn == b.bin) list_add(col, l);
      if (!from_hist && bn < b.bin) {
        const uint64_t w = weight(l);
        if (w >= minw) sum += w;
      }
    });
    uint32_t cnt = list_send(buf, block_sum(sum));
    if (cnt <= (uint32_t)kList) {
      list_weigh((int)cnt);
      list_border((int)cnt, (float)b.bin, (float)kBins, b.n_above, b.m_above, target, by_mass);
      return (int)cnt;
    }
    // too many: split the bin, then send what is left of it
    refine(b, target, by_mass);
    const bool one_key = b.n_in > (uint32_t)kList;
    sum = 0;
    each([&](int col, float l) {
      const float ph = lead(l);
      if (!alive(ph) || bin_of(ph) > b.bin) return;
      bool sure = bin_of(ph) < b.bin;
      if (!sure) {
        const uint64_t k = key_of(l, col);
        if (k < b.klo) return;
        sure = one_key || k > b.khi;
      }
      if (!sure) {
        list_add(col, l);
      } else {
        const uint64_t w = weight(l);
        if (w >= minw) sum += w;
      }
    });
    __syncthreads();
    if (tid == 0) sh.ltotal[buf] = 0;
    cl.sync();  // every block has cleared its total and is done with the first list
    cnt = list_send(buf, block_sum(sum));
    if (one_key) return 0;
    list_weigh((int)cnt);
    list_border((int)cnt, (float)b.bin, (float)kBins, b.n_above, b.m_above, target, by_mass);
    return (int)cnt;
  }

  // The block's least and largest, in every thread.
  __device__ void block_range(uint64_t& lo, uint64_t& hi) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = min(lo, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)lo, o));
      hi = max(hi, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)hi, o));
    }
    __syncthreads();
    if (lane == 0) {
      sh.w64[warp] = lo;
      sh.x64[warp] = hi;
    }
    __syncthreads();
    for (int w = 0; w < kW; ++w) {
      lo = min(lo, sh.w64[w]);
      hi = max(hi, sh.x64[w]);
    }
  }

  // Sum over the block, in every thread; the warps' sums stay in wsum.
  __device__ uint64_t block_sum(uint64_t v) {
    v = warp_sum64(v);
    __syncthreads();
    if (lane == 0) sh.wsum[warp] = v;
    __syncthreads();
    uint64_t t = 0;
#pragma unroll
    for (int w = 0; w < kW; ++w) t += sh.wsum[w];
    return t;
  }

  __device__ void nothing() {  // no column to draw from, or bad parameters
    if (rank == 0 && tid == 0) {
      a.ids[(int64_t)row * a.ldt] = -1;
      if (a.prob) a.prob[(int64_t)row * a.ldt] = 0.0f;
    }
    if (a.probs)
      each([&](int col, float) {
        if (col >= 0 && col < n) a.probs[(int64_t)row * a.ldp + col] = 0.0f;
      });
  }

  __device__ void run() {
    if (tid < 128) sh.tab[tid] = kExp2Table[tid];
    if (tid < 2) sh.ltotal[tid] = 0;
    if (tid == 2) sh.n_out = 0;
    hist_zero();
    cl.barrier_arrive();  // waited for in extremes()
    float t = a.temperature ? a.temperature[row] : 1.0f;
    int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    const float minp = a.min_p ? a.min_p[row] : 0.0f;
    const float u = a.u[row];
    const bool good = t >= 0.0f && t < INFINITY && p == p && minp == minp && u >= 0.0f && u < 1.0f;
    if (t == 0.0f) {
      t = 1.0f;
      k = 1;
    }
    float mn, mt, own;
    extremes(mn, mt, own);
    if (!good && rank == 0 && tid == 0) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
    if (!good || m == -INFINITY) {
      nothing();
      return;
    }
    if (m == INFINITY) {
      inf = true;
      m = mn = 0.0f;
      mt = 0.0f;
      own = own == INFINITY ? 0.0f : -INFINITY;
      if (KEEP)
        for (int v = vbeg + lane; v < vend; v += 32) keep[v - vcta] = only_inf(keep[v - vcta]);
    }
    sc = scale_of(t);
    const float mp = fminf(fmaxf(minp, 0.0f), 1.0f);
    minw = __float2ull_ru(mp * 8796093022208.0f);
    log2_minp = minw ? __log2f(mp) : 0.0f;
    lfloor = logit_at(fmaxf(kCutLog2, minw ? log2_minp - 1e-3f : kCutLog2), true);
    const bool use_k = k > 0 && k < n, use_p = p < 1.0f;
    uint64_t tkey = 0;
    int buf = 0, ncand = 0;
    bool all_listed = false;  // every kept column is in the list

    auto p_target = [&](uint64_t z) {
      return max((uint64_t)1, mul_frac(fmaxf(p, 0.0f), z, true));
    };
    auto spread = [&](float lowest, float cut) {  // bins from the largest logit to this one or the cut
      const float span = fminf(-lead(lowest) * 1.0001f, 0.01f - cut);
      binscale = (float)kBins / fmaxf(span, 1e-30f);
    };

    bool open = use_k || use_p;  // a filter is left to resolve
    if (use_k && k <= kList && (int64_t)k <= (int64_t)kT * C) {
      spread(mt, kCutLog2);
      const float ph = lead(own);
      const int mine = alive(ph) ? bin_of(ph) : kBins;
      if (mine < kBins) atomicAdd(&sh.cnt[mine], 1u);
      hist_sum(true, false);
      zero_masses();
      const int b = find((uint64_t)k, false, 0, 0);
      if (b < kBins) {
        if (mine <= b)
          for (int v = vbeg + lane; v < vend; v += 32) {
            const uint4 r = get(v);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
              const float l = elem(r, j), q = lead(l);
              if (alive(q) && bin_of(q) <= b) list_add(v * VE + j - off, l);
            }
          }
        const uint32_t cnt = list_send(0, 0);
        if (cnt <= (uint32_t)kList) {
          ncand = (int)cnt;
          list_weigh(ncand);
          const float mul = (float)kBins / (float)(b + 1);
          list_border(ncand, 0.0f, mul, 0, 0, (uint64_t)k, false);
          if (use_p) {
            const uint64_t zk = sh.zk;
            __syncthreads();  // every thread has read it: a short list is ranked, and zk written, at once
            list_border(ncand, 0.0f, mul, 0, 0, p_target(zk), true);
          }
          tkey = sh.tkey;
          all_listed = true;
          open = false;
        }
      }
      if (open) {  // the columns' own histogram, from scratch
        buf = 1;
        __syncthreads();
        hist_zero();
        __syncthreads();
      }
    }
    if (open) {
      // top-p alone: the columns of a weight under 2^-20 add up to under 2^-20 n, seldom more than
      // the share that top-p cuts off
      float cut = use_k ? kCutLog2 : -20.0f;
      spread(mn, cut);
      uint64_t tail = hist_row(use_k, use_p, cut);
      if (!use_k) zero_counts();
      if (!use_p) zero_masses();
      uint32_t total = 0;
      uint64_t z = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        total += sh.rcnt[tid * kPer + i];
        z += sh.rmass[tid * kPer + i];
      }
      z = block_sum(z);
      if (use_k) total = (uint32_t)block_sum(total);
      const bool by_k = use_k && total > (uint32_t)k;
      bool again = false;  // the histogram has to be taken once more
      if (by_k) {
        const uint64_t given = minw;
        if (use_p) minw = 0;  // top-p goes by the mass of all columns that top-k leaves
        ncand = row_border(buf, (uint64_t)k, false, use_p);
        if (use_p) minw = given;
        tkey = sh.tkey;
        z = sh.zk;
        again = use_p;
      }
      if (use_p) {
        if (!by_k) {
          again = p_target(z + tail) > z;  // the border lies below the cut
          z += tail;
        }
        if (again) {
          __syncthreads();
          hist_zero();
          if (tid == 0) sh.ltotal[buf] = 0;
          cl.sync();
          spread(mn, kCutLog2);
          hist_row(false, true, kCutLog2);
          zero_counts();
        }
        ncand = row_border(buf, p_target(z), true, true);
        tkey = sh.tkey;
      }
      open = by_k || use_p;
      if (ncand < 0) {  // min_p is the stricter one
        ncand = 0;
        tkey = 0;
        open = false;
      }
    }
    if (!all_listed && !open) {  // everything that min_p keeps
      uint64_t sum = 0;
      if (minw) {
        sum = lane_share<KEEP>(vbeg, vend, -INFINITY, 0);
      } else {
        for (int v = vbeg + lane; v < vend; v += 32) {
          const uint4 r = get(v);
          bool any = false;
#pragma unroll
          for (int j = 0; j < VE; ++j) any |= elem(r, j) >= lfloor;
          if (!any) continue;
#pragma unroll
          for (int j = 0; j < VE; ++j) sum += weight(elem(r, j));
        }
      }
      sum = block_sum(sum);
      if (tid < C) *cl.map_shared_rank(&sh.cdef[buf][rank], tid) = sum;
      cl.sync();
    }

    // the kept mass of every block, and of this block's warps
    if (tid < kMaxC * 3) (&sh.cw3[0][0])[tid] = 0u;
    if (tid < kW * 3) (&sh.ww3[0][0])[tid] = 0u;
    __syncthreads();
    for (int i = tid; i < ncand; i += kT) {
      const uint64_t w = sh.lw[i];
      if (sh.lkey[i] >= tkey && w >= minw) {
        const int v = ((int)(uint32_t)sh.lent[i] + off) / VE, c = v / nvc;
        pieces_add(&sh.cw3[0][c], &sh.cw3[1][c], &sh.cw3[2][c], w);
        if (c == rank) {
          const int q = (v - vcta) / nvw;
          pieces_add(&sh.ww3[0][q], &sh.ww3[1][q], &sh.ww3[2][q], w);
        }
      }
    }
    __syncthreads();
    auto block_mass = [&](int c) {
      return (all_listed ? 0 : sh.cdef[buf][c]) +
             pieces(sh.cw3[0][c], sh.cw3[1][c], sh.cw3[2][c]);
    };
    uint64_t z = 0, before = 0;
    for (int c = 0; c < C; ++c) z += block_mass(c);
    const uint64_t target = mul_frac(u, z, false);
    int owner = 0;  // the block that holds the drawn column
    for (; owner < C - 1; ++owner) {
      const uint64_t x = block_mass(owner);
      if (target < before + x) break;
      before += x;
    }
    const float zf = 1.0f / (__ull2float_rn(z) * (1.0f / 8796093022208.0f));
    const float tval = tkey ? key_value(tkey) : -INFINITY;
    lfloor = fmaxf(lfloor, tval);
    // Way C: the kept masses of that block's warps, column by column: a share by every block (96 x 163840
    // with top-p 0.9: 116 us by that block alone, 107 so).
    if (open) {
      const int v0 = owner * nvc + warp * nvw;
      const int v1 = min(min(v0 + nvw, owner * nvc + nvc), nvrow);
      const int per = (max(v1 - v0, 0) + C - 1) / C, from = v0 + rank * per;
      const uint64_t sum = warp_sum64(lane_share<false>(from, min(from + per, v1), tval, tkey));
      if (lane == 0) *cl.map_shared_rank(&sh.part[rank][warp], owner) = sum;
      cl.sync();
      if (tid < kW) {
        uint64_t t = 0;
        for (int c = 0; c < C; ++c) t += sh.part[c][tid];
        sh.wsum[tid] = t;
      }
      __syncthreads();
    }
    if (rank == owner) {
      uint64_t ws = 0;  // the warp whose columns hold it
      if (lane < kW)
        ws = all_listed ? pieces(sh.ww3[0][lane], sh.ww3[1][lane], sh.ww3[2][lane]) : sh.wsum[lane];
      uint64_t incl = ws;
#pragma unroll
      for (int o = 1; o < kW; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, (unsigned long long)incl, o);
        if (lane >= o) incl += x;
      }
      const int w = __ffs(__ballot_sync(0xffffffffu, before + incl > target)) - 1;
      before += __shfl_sync(0xffffffffu, (unsigned long long)(incl - ws), w);
      const int v = vcta + w * nvw;
      search(v, min(min(v + nvw, vcta + nvc), nvrow), before, target, tval, tkey, zf);
    }
    if (a.probs) write_probs(tval, tkey, zf);
  }

  __device__ __forceinline__ bool above(float l, int col, float tval, uint64_t tkey) const {
    return l > tval || (l == tval && key_of(l, col) >= tkey);
  }
  // The kept weights of 16 bytes of columns, and their sum.
  __device__ __forceinline__ uint64_t kept_weights(int v, float tval, uint64_t tkey,
                                                   uint64_t (&w)[VE]) const {
    const uint4 r = get(v);
    uint64_t sum = 0;
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      const float l = elem(r, j);
      uint64_t x = 0;
      if (l >= lfloor && above(l, v * VE + j - off, tval, tkey)) {
        x = weight(l);
        if (x < minw) x = 0;
      }
      w[j] = x;
      sum += x;
    }
    return sum;
  }

  // This lane's share of the kept mass of the 16-byte pieces from beg to end, which are the warp's (of
  // this block's own columns or another's). Kept columns are few as a rule, so they queue in shared
  // memory (the histogram's, done with) and are weighed 32 at a time (96 x 163840: 148 to 140 us).
  template <bool OWN>
  __device__ __forceinline__ uint64_t lane_share(int beg, int end, float tval, uint64_t tkey) {
    float* queue = reinterpret_cast<float*>(sh.w.lo) + warp * 64;
    uint64_t sum = 0;
    int cnt = 0;
#pragma unroll 1
    for (int v0 = beg; v0 < end; v0 += 32) {
      const int v = v0 + lane;
      const uint32_t none = BF16 ? 0x7FC07FC0u : 0x7FC00000u;
      uint4 r = make_uint4(none, none, none, none);
      if (v < end) {
        if (OWN) {
          r = get(v);
        } else {
          r = load(v);
          if (inf) r = only_inf(r);
        }
      }
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float l = elem(r, j);
        const bool on = l >= lfloor && above(l, v * VE + j - off, tval, tkey);
        const unsigned who = __ballot_sync(0xffffffffu, on);
        if (on) queue[cnt + __popc(who & ((1u << lane) - 1))] = l;
        cnt += __popc(who);
        if (cnt >= 32) {
          __syncwarp();
          const uint64_t w = weight(queue[cnt - 32 + lane]);
          sum += w >= minw ? w : 0;
          cnt -= 32;
          __syncwarp();
        }
      }
    }
    __syncwarp();
    if (lane < cnt) {
      const uint64_t w = weight(queue[lane]);
      sum += w >= minw ? w : 0;
    }
    return sum;
  }

  // The block, over the 16-byte pieces of one warp's columns: the first column whose running kept
  // mass exceeds the target. A piece a thread, so it takes one step or two where that warp alone
  // would take many.
  __device__ void search(int v0, int v1, uint64_t before, uint64_t target, float tval,
                         uint64_t tkey, float zf) {
#pragma unroll 1
    for (; v0 < v1; v0 += kT) {
      const int v = v0 + tid;
      uint64_t w[VE], sum = 0;
#pragma unroll
      for (int j = 0; j < VE; ++j) w[j] = 0;
      if (v < v1) sum = kept_weights(v, tval, tkey, w);
      uint64_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, (unsigned long long)incl, o);
        if (lane >= o) incl += x;
      }
      __syncthreads();
      if (lane == 31) sh.w64[warp] = incl;
      __syncthreads();
      const uint64_t mine = lane < kW ? sh.w64[lane] : 0;
      uint64_t run = before + warp_sum64(lane < warp ? mine : 0) + incl - sum;
      before += warp_sum64(mine);
      if (run <= target && run + sum > target) {
        bool done = false;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          run += w[j];
          if (!done && run > target) {
            done = true;
            const int col = v * VE + j - off;
            const float l = elem(get(v), j);
            a.ids[(int64_t)row * a.ldt] = a.id_map ? a.id_map[col] : col;
            if (a.prob) a.prob[(int64_t)row * a.ldt] = weight_float(l, m, sc, lead(l)) * zf;
          }
        }
      }
      if (before > target) return;
    }
  }

  __device__ void write_probs(float tval, uint64_t tkey, float zf) {
    float* out = a.probs + (int64_t)row * a.ldp;
    const bool vec = (((uintptr_t)(out - off)) & 15) == 0;
    for (int v = vbeg + lane; v < vend; v += 32) {
      const uint4 r = get(v);
      float q[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float l = elem(r, j);
        q[j] = 0.0f;
        if (l >= lfloor && above(l, v * VE + j - off, tval, tkey)) {
          const float ph = lead(l);
          if (alive(ph) && (minw == 0 || weight(l) >= minw)) q[j] = weight_float(l, m, sc, ph) * zf;
        }
      }
      const int c0 = v * VE - off;
      if (vec && c0 >= 0 && c0 + VE <= n) {
#pragma unroll
        for (int j = 0; j < VE; j += 4)
          *(float4*)(out + c0 + j) = make_float4(q[j], q[j + 1], q[j + 2], q[j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (c0 + j >= 0 && c0 + j < n) out[c0 + j] = q[j];
      }
    }
  }
};

template <bool BF16, bool KEEP>
__global__ void __launch_bounds__(kT, 2) sample_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char smem[];
  tfd_host::after_previous();
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  uint4* keep = reinterpret_cast<uint4*>(smem + ((sizeof(Shared) + 15) / 16) * 16);
  Sampler<BF16, KEEP> s(a, sh, keep);
  s.run();
}

}  // namespace

extern "C" tfd_status tfd_sample(const void* logits, int lfmt, int rows, int64_t n, int64_t ld,
                                 const float* temperature, const int32_t* top_k,
                                 const float* top_p, const float* min_p, const float* u,
                                 const int32_t* id_map, int32_t* ids, float* prob, int64_t ldt,
                                 float* probs, int64_t ldp, int32_t* dev_status, void* stream) {
  using tfd_host::aligned;
  if (!logits || !u || !ids) return TFD_ERR_INVALID;
  if (lfmt != TFD_X_BF16 && lfmt != TFD_X_F32) return TFD_ERR_INVALID;
  if (rows < 1 || n < 1 || ld < n || ldt < 0 || (probs && ldp < n)) return TFD_ERR_INVALID;
  if (n > kMaxDrawCols || rows > (1 << 24)) return TFD_ERR_UNSUPPORTED;
  if (!aligned(logits, lfmt == TFD_X_BF16 ? 2 : 4) || (probs && !aligned(probs, 4)))
    return TFD_ERR_INVALID;
  for (const void* p : {(const void*)temperature, (const void*)top_k, (const void*)top_p,
                        (const void*)min_p, (const void*)u, (const void*)id_map,
                        (const void*)ids, (const void*)prob, (const void*)dev_status})
    if (p && !aligned(p, 4)) return TFD_ERR_INVALID;
  if (ldt == 0) ldt = 1;
  const bool bf16 = lfmt == TFD_X_BF16;
  const int es = bf16 ? 2 : 4, ve = 16 / es;
  // outputs apart from the inputs: a row's blocks read them for themselves
  const int64_t last = (int64_t)rows - 1, four = (int64_t)rows * 4;
  const struct { const void* p; int64_t bytes; } outs[] = {
      {ids, (last * ldt + 1) * 4}, {prob, (last * ldt + 1) * 4}, {probs, (last * ldp + n) * 4}},
      ins[] = {{logits, (last * ld + n) * es}, {temperature, four}, {top_k, four}, {top_p, four},
               {min_p, four}, {u, four}, {id_map, n * 4}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (tfd_host::overlap(o.p, o.bytes, i.p, i.bytes)) return TFD_ERR_INVALID;

  const int64_t nv = (n + ve - 1) / ve + 1;  // one more where a row starts off a 16-byte boundary
  const size_t fixed = (sizeof(Shared) + 15) / 16 * 16;
  int dev = 0;
  tfd_host::device_sms(dev);
  // Blocks a row. A launch runs in rounds of as many clusters as fit at two blocks an SM; a round
  // costs about as much as 16384 columns besides its blocks' own, and columns that do not fit shared
  // memory beside another block's are read from L2 by every pass, for about 0.4 of their time more.
  auto part = [&](int blocks) { return (size_t)((nv + blocks - 1) / blocks + 1) * 16; };
  const size_t half = 112 * 1024;
  if (!tfd_host::allow_clusters<sample_kernel<false, true>>(dev, tfd_host::kSmemLimit))
    return TFD_ERR_CUDA;
  const int c = tfd_host::cheapest_cluster(
      rows,
      [&](int i) {
        return tfd_host::clusters_at_once<sample_kernel<false, true>>(dev, i, kT, half);
      },
      [&](int i) { return i == kMaxC || n / i < kMaxPart; },
      [&](int i, int64_t rounds) {
        const int64_t cols = n / i, own = fixed + part(i) <= half ? cols : cols * 14 / 10;
        return rounds * (16384 + 256 * i + own);
      });
  if (c == 0) return TFD_ERR_UNSUPPORTED;
  const bool keep = fixed + part(c) <= half;
  const size_t smem = fixed + (keep ? part(c) : 0);
  Args a = {logits, n, ld, temperature, top_k, top_p, min_p, u, id_map, ids, prob, ldt, probs, ldp,
            dev_status};
  cudaStream_t st = tfd_host::as_stream(stream);
#define TFD_SAMPLE_CASE(B, K)                                                        \
  if (bf16 == B && keep == K)                                                        \
    return tfd_host::launch_clusters<sample_kernel<B, K>>(a, dev, rows, c, kT, smem, \
                                                          tfd_host::kSmemLimit, st);
  TFD_SAMPLE_CASE(true, true) TFD_SAMPLE_CASE(true, false)
  TFD_SAMPLE_CASE(false, true) TFD_SAMPLE_CASE(false, false)
#undef TFD_SAMPLE_CASE
  return TFD_ERR_UNSUPPORTED;
}
