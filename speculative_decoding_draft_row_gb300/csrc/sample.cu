// sample.cu - draws one token a row from its logits and a given random number, after temperature,
// top-k, top-p and min-p, optionally with the whole filtered distribution.
//
// Weights are exact integers (weight.cuh), so a row's sums are the same in any order. One
// thread-block cluster takes a row, each block a contiguous part of its columns, each warp a
// contiguous part of the block's. The steps, with a cluster barrier after each of 1 to 4:
//  1. the row's largest and smallest finite logit;
//  2. with top-k or top-p: a histogram of the columns over log2 of their weight (2048 bins from
//     the largest down to the smallest or to the 2^-44 cut; counts, and masses where top-p asks);
//  3. the blocks' histograms summed, an eighth of the bins or so by each block, into every block;
//  4. the bin in which the border falls is found by each block on its own; the columns above it
//     are kept for certain and their mass summed per warp, the few columns inside it are sent to
//     every block, which ranks them and knows the last kept (value, id) key;
//  5. every block knows all blocks' kept masses, so the one that holds the drawn column finds its
//     warp, and that warp scans its columns for it.
// A bin with more columns than the candidate list holds is split again by the columns' 64-bit keys
// until it fits (equal logits differ by their ids, so this ends). Without top-k and top-p steps 2
// and 3 fall away.
#include <cooperative_groups.h>

#include "launch.cuh"
#include "weight.cuh"

namespace {

using namespace tfd;
namespace cg = cooperative_groups;

constexpr int kT = 512;
constexpr int kW = kT / 32;
constexpr int kBins = 2048;
constexpr int kPer = kBins / kT;
constexpr int kCand = 256;
constexpr int kMaxC = 16;

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

struct Shared {
  unsigned long long tab[128];
  uint32_t cnt[kBins], mlo[kBins], mhi[kBins];  // this block's histogram
  uint32_t rcnt[kBins];                         // the row's
  uint64_t rmass[kBins];
  uint64_t ckey[2][kCand], cw[2][kCand];  // candidates of the border bin, in every block
  uint32_t ccol[2][kCand];
  uint32_t ccount[2];                     // rank 0: candidates appended
  float cmax[kMaxC], cmin[kMaxC];
  uint64_t cdef[2][kMaxC];                // mass of each block's columns above the border bin
  uint64_t klo[kMaxC], khi[kMaxC];
  uint64_t wdef[kW];                      // the same of this block's warps
  uint64_t cmass[kMaxC];
  uint64_t w64[kW];
  uint32_t w32[kW];
  float wmax[kW], wmin[kW];
  uint64_t f_above_m, f_in_m, tkey, zk;
  uint32_t f_bin, f_above_n, f_in_n;
};

// The border of a filter: columns in bins below `bin` (higher weights) are kept for certain, and
// of `bin` itself those with a key above khi; keys in [klo, khi] are undecided.
struct Border {
  int bin;
  uint64_t klo, khi;
  uint32_t n_above, n_in;
  uint64_t m_above, m_in;
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
  int C, rank, row, off, n, nvc, nvw, vcta, vbeg, vend;
  const char* base;
  // the row's parameters
  float m, binscale, minp;
  Scale sc;
  uint64_t minw;

  __device__ Sampler(const Args& args, Shared& s, uint4* kp) : a(args), sh(s), keep(kp) {
    C = (int)cl.num_blocks();
    rank = (int)cl.block_rank();
    row = blockIdx.x / C;
    n = (int)a.n;
    const int es = BF16 ? 2 : 4;
    const char* p = (const char*)a.logits + (int64_t)row * a.ld * es;
    off = (int)((uintptr_t)p & 15) / es;
    base = p - off * es;
    const int nv = (off + n + VE - 1) / VE;
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
  __device__ __forceinline__ uint4 get(int v) const { return KEEP ? keep[v - vcta] : load(v); }
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

  __device__ __forceinline__ float lead(float l) const { return lead_log2(l, m, sc); }
  __device__ __forceinline__ int bin_of(float ph) const {
    return min(kBins - 1, (int)(-ph * binscale));
  }
  __device__ __forceinline__ uint64_t weight(float l, float ph) const {
    int e;
    const uint64_t t = weight_mant(l, m, sc, ph, sh.tab, e);
    return weight_fix(t, e);
  }
  __device__ __forceinline__ uint64_t key_of(float l, int col) const {
    return make_key(l, a.id_map ? a.id_map[col] : col);
  }
  __device__ __forceinline__ bool at_least(float l, int col, uint64_t tkey) const {
    const uint32_t vk = value_key(l), th = (uint32_t)(tkey >> 32);
    return vk != th ? vk > th : key_of(l, col) >= tkey;
  }

  __device__ void extremes(float& mn) {
    float mx = -INFINITY;
    mn = INFINITY;
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
            if (x > -INFINITY) mn = fminf(mn, x);
          }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    }
    if (lane == 0) {
      sh.wmax[warp] = mx;
      sh.wmin[warp] = mn;
    }
    __syncthreads();
    if (tid < C) {  // the other blocks run: barrier of the constructor's caller
      for (int w = 0; w < kW; ++w) {
        mx = fmaxf(mx, sh.wmax[w]);
        mn = fminf(mn, sh.wmin[w]);
      }
      *cl.map_shared_rank(&sh.cmax[rank], tid) = mx;
      *cl.map_shared_rank(&sh.cmin[rank], tid) = mn;
    }
    cl.sync();
    m = sh.cmax[0];
    mn = sh.cmin[0];
    for (int c = 1; c < C; ++c) {
      m = fmaxf(m, sh.cmax[c]);
      mn = fminf(mn, sh.cmin[c]);
    }
  }

  __device__ __forceinline__ void hist_add(int b, uint64_t w, bool mass) {
    atomicAdd(&sh.cnt[b], 1u);
    if (mass) {  // a 64-bit sum in two words, the carry taken from the low word's old value
      const uint32_t lo = (uint32_t)w;
      const uint32_t old = atomicAdd(&sh.mlo[b], lo);
      const uint32_t hi = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
      if (hi) atomicAdd(&sh.mhi[b], hi);
    }
  }
  __device__ void hist_zero() {
    for (int b = tid; b < kBins; b += kT) sh.cnt[b] = sh.mlo[b] = sh.mhi[b] = 0u;
    __syncthreads();
  }
  // The blocks' histograms summed into every block's rcnt, rmass.
  __device__ void hist_sum() {
    cl.sync();
    const int per = kBins / C;
    for (int i = tid; i < per; i += kT) {
      const int b = rank * per + i;
      uint32_t c = 0;
      uint64_t w = 0;
      for (int r = 0; r < C; ++r) {
        c += *cl.map_shared_rank(&sh.cnt[b], r);
        w += *cl.map_shared_rank(&sh.mlo[b], r) +
             ((uint64_t)*cl.map_shared_rank(&sh.mhi[b], r) << 32);
      }
      for (int r = 0; r < C; ++r) {
        *cl.map_shared_rank(&sh.rcnt[b], r) = c;
        *cl.map_shared_rank(&sh.rmass[b], r) = w;
      }
    }
    cl.sync();
  }
  __device__ void hist_rows(bool mass) {
    hist_zero();
    each([&](int, float l) {
      const float ph = lead(l);
      if (alive(ph)) hist_add(bin_of(ph), mass ? weight(l, ph) : 0, mass);
    });
    hist_sum();
  }

  // The first bin at which the running count (or mass) from bin 0 reaches `target`; false if none.
  __device__ bool find(uint64_t target, bool by_mass, uint32_t n0, uint64_t m0, Border& b) {
    uint32_t c = 0;
    uint64_t w = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c += sh.rcnt[tid * kPer + i];
      w += sh.rmass[tid * kPer + i];
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
    __syncthreads();
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
      const uint32_t cn = sh.rcnt[tid * kPer + i];
      const uint64_t wn = sh.rmass[tid * kPer + i];
      const uint64_t before = by_mass ? wb : cb, after = by_mass ? wb + wn : cb + cn;
      if (before < target && after >= target) {
        sh.f_bin = tid * kPer + i;
        sh.f_above_n = cb;
        sh.f_above_m = wb;
        sh.f_in_n = cn;
        sh.f_in_m = wn;
      }
      cb += cn;
      wb += wn;
    }
    __syncthreads();
    b.bin = (int)sh.f_bin;
    b.klo = 0;
    b.khi = ~0ull;
    b.n_above = sh.f_above_n;
    b.m_above = sh.f_above_m;
    b.n_in = sh.f_in_n;
    b.m_in = sh.f_in_m;
    return b.bin < kBins;
  }

  // Splits the border's bin by its columns' keys until the undecided columns fit the list, or have
  // one key. Overwrites the histogram; returns whether it did.
  __device__ bool refine(Border& b, uint64_t target, bool by_mass, bool mass) {
    bool did = false;
    const int bin = b.bin;
    while (b.n_in > kCand && b.klo < b.khi) {
      did = true;
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
        sh.cmass[warp] = hi;  // free until the draw
      }
      __syncthreads();
      if (tid < C) {
        for (int w = 0; w < kW; ++w) {
          lo = min(lo, sh.w64[w]);
          hi = max(hi, sh.cmass[w]);
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
      const int shift = max(0, 64 - __clzll((long long)span) - 11);  // (span >> shift) < 2048
      each([&](int col, float l) {
        const float ph = lead(l);
        if (alive(ph) && bin_of(ph) == bin) {
          const uint64_t k = key_of(l, col);
          if (k >= lo && k <= hi) hist_add((int)((hi - k) >> shift), mass ? weight(l, ph) : 0, mass);
        }
      });
      hist_sum();
      Border s;
      find(target, by_mass, b.n_above, b.m_above, s);
      b.n_above = s.n_above;
      b.m_above = s.m_above;
      b.n_in = s.n_in;
      b.m_in = s.m_in;
      b.khi = hi - ((uint64_t)s.bin << shift);
      const uint64_t width = (1ull << shift) - 1;
      b.klo = b.khi - lo < width ? lo : b.khi - width;
    }
    b.bin = bin;
    return did;
  }

  // Sums the kept-for-certain columns' masses and sends the undecided ones to every block.
  __device__ void gather(int buf, const Border& b) {
    const bool collapsed = b.n_in > kCand;  // one key: all of it is kept
    uint64_t sum = 0;
    each([&](int col, float l) {
      const float ph = lead(l);
      if (!alive(ph)) return;
      const int bn = bin_of(ph);
      if (bn > b.bin) return;
      const uint64_t w = weight(l, ph);
      uint64_t k = 0;
      bool sure = bn < b.bin;
      if (!sure) {
        k = key_of(l, col);
        if (k < b.klo) return;
        sure = collapsed || k > b.khi;
      }
      if (sure) {
        if (w >= minw) sum += w;
        return;
      }
      const uint32_t slot = atomicAdd(cl.map_shared_rank(&sh.ccount[buf], 0), 1u);
      for (int r = 0; r < C; ++r) {
        *cl.map_shared_rank(&sh.ckey[buf][slot], r) = k;
        *cl.map_shared_rank(&sh.cw[buf][slot], r) = w;
        *cl.map_shared_rank(&sh.ccol[buf][slot], r) = (uint32_t)col;
      }
    });
    sum = warp_sum64(sum);
    if (lane == 0) sh.wdef[warp] = sum;
    __syncthreads();
    if (tid < C) {
      uint64_t t = 0;
      for (int w = 0; w < kW; ++w) t += sh.wdef[w];
      *cl.map_shared_rank(&sh.cdef[buf][rank], tid) = t;
    }
    cl.sync();
  }

  // The last kept key among the candidates: the need-th column, or the one whose running mass
  // reaches the target. Also the mass up to and with it.
  __device__ void resolve(int buf, const Border& b, uint64_t target, bool by_mass) {
    if (b.n_in > kCand) {
      __syncthreads();
      if (tid == 0) {
        sh.tkey = b.klo;
        sh.zk = b.m_above + b.m_in;
      }
      __syncthreads();
      return;
    }
    __syncthreads();
    for (int i = tid; i < (int)b.n_in; i += kT) {
      const uint64_t k = sh.ckey[buf][i], w = sh.cw[buf][i];
      const uint32_t col = sh.ccol[buf][i];
      uint32_t above = b.n_above;
      uint64_t before = b.m_above;
      for (int j = 0; j < (int)b.n_in; ++j) {
        const uint64_t kj = sh.ckey[buf][j];
        if (kj > k || (kj == k && sh.ccol[buf][j] < col)) {
          ++above;
          before += sh.cw[buf][j];
        }
      }
      const bool hit = by_mass ? (before < target && before + w >= target)
                               : (uint64_t)above + 1 == target;
      if (hit) {
        sh.tkey = k;
        sh.zk = before + w;
      }
    }
    __syncthreads();
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
    if (tid < 2) sh.ccount[tid] = 0;
    float t = a.temperature ? a.temperature[row] : 1.0f;
    int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    minp = a.min_p ? a.min_p[row] : 0.0f;
    const float u = a.u[row];
    const bool good = t >= 0.0f && t < INFINITY && p == p && minp == minp && u >= 0.0f && u < 1.0f;
    if (t == 0.0f) {
      t = 1.0f;
      k = 1;
    }
    cl.sync();  // every block runs and has cleared its counters
    float mn;
    extremes(mn);
    if (!good && rank == 0 && tid == 0) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
    if (!good || m == -INFINITY) {
      nothing();
      return;
    }
    sc = scale_of(t);
    minw = __float2ull_ru(fminf(fmaxf(minp, 0.0f), 1.0f) * 8796093022208.0f);
    const bool use_k = k > 0 && k < n, use_p = p < 1.0f;
    uint64_t tkey = 0;
    int buf = 0, ncand = 0;
    if (use_k || use_p) {
      const float span = fminf(-lead(mn) * 1.0001f, -kCutLog2 + 0.01f);
      binscale = (float)kBins / fmaxf(span, 1e-30f);
      hist_rows(use_p);
      Border bk, bp;
      bool gathered = false, dirty = false;
      uint64_t zk = 0;
      if (use_k && find((uint64_t)k, false, 0, 0, bk)) {
        dirty = refine(bk, (uint64_t)k, false, use_p);
        gather(0, bk);
        resolve(0, bk, (uint64_t)k, false);
        tkey = sh.tkey;
        zk = sh.zk;
        gathered = true;
        ncand = bk.n_in > kCand ? 0 : (int)bk.n_in;
      } else if (use_p) {
        uint64_t w = 0;
        for (int i = 0; i < kPer; ++i) w += sh.rmass[tid * kPer + i];
        w = warp_sum64(w);
        __syncthreads();
        if (lane == 0) sh.w64[warp] = w;
        __syncthreads();
        for (int q = 0; q < kW; ++q) zk += sh.w64[q];
      }
      if (use_p) {
        const uint64_t target = max((uint64_t)1, mul_frac(fmaxf(p, 0.0f), zk, true));
        if (dirty) hist_rows(true);
        find(target, true, 0, 0, bp);
        const bool split = refine(bp, target, true, true);
        if (!gathered || dirty || split || bp.bin != bk.bin) {
          buf = gathered ? 1 : 0;
          gather(buf, bp);
          ncand = bp.n_in > kCand ? 0 : (int)bp.n_in;
        }
        resolve(buf, bp, target, true);
        tkey = sh.tkey;
        gathered = true;
      }
      if (!gathered) {
        Border all = {kBins, 0, ~0ull, 0, 0, 0, 0};
        gather(0, all);
      }
    } else {
      binscale = 0.0f;
      Border all = {kBins, 0, ~0ull, 0, 0, 0, 0};
      gather(0, all);
    }

    // kept mass of every block, and of this block's warps
    __syncthreads();
    if (tid < C) sh.cmass[tid] = sh.cdef[buf][tid];
    __syncthreads();
    for (int i = tid; i < ncand; i += kT) {
      if (sh.ckey[buf][i] >= tkey && sh.cw[buf][i] >= minw) {
        const int v = ((int)sh.ccol[buf][i] + off) / VE, c = v / nvc;
        atomicAdd((unsigned long long*)&sh.cmass[c], (unsigned long long)sh.cw[buf][i]);
        if (c == rank)
          atomicAdd((unsigned long long*)&sh.wdef[(v - vcta) / nvw],
                    (unsigned long long)sh.cw[buf][i]);
      }
    }
    __syncthreads();
    uint64_t z = 0;
    for (int c = 0; c < C; ++c) z += sh.cmass[c];
    const uint64_t target = mul_frac(u, z, false);
    const float zf = 1.0f / (__ull2float_rn(z) * (1.0f / 8796093022208.0f));
    uint64_t before = 0;
    for (int c = 0; c < rank; ++c) before += sh.cmass[c];
    if (target >= before && target < before + sh.cmass[rank]) {
      for (int w = 0; w < warp; ++w) before += sh.wdef[w];
      if (target >= before && target < before + sh.wdef[warp]) search(before, target, tkey, zf);
    }
    if (a.probs) write_probs(tkey, zf);
  }

  // One warp: the first of its columns whose running kept mass exceeds the target.
  __device__ void search(uint64_t before, uint64_t target, uint64_t tkey, float zf) {
    for (int v0 = vbeg; v0 < vend; v0 += 32) {
      const int v = v0 + lane;
      uint64_t w[VE], sum = 0;
      uint4 r = make_uint4(0, 0, 0, 0);
      if (v < vend) r = get(v);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        w[j] = 0;
        if (v < vend) {
          const float l = elem(r, j);
          const float ph = lead(l);
          if (alive(ph) && at_least(l, v * VE + j - off, tkey)) {
            const uint64_t x = weight(l, ph);
            if (x >= minw) w[j] = x;
          }
        }
        sum += w[j];
      }
      uint64_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, (unsigned long long)incl, o);
        if (lane >= o) incl += x;
      }
      const uint64_t total = __shfl_sync(0xffffffffu, (unsigned long long)incl, 31);
      if (before + total > target) {
        uint64_t run = before + incl - sum;
        if (run <= target && before + incl > target) {
          bool done = false;
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            run += w[j];
            if (!done && run > target) {
              done = true;
              const int col = v * VE + j - off;
              const float l = elem(r, j);
              int e;
              const uint64_t mant = weight_mant(l, m, sc, lead(l), sh.tab, e);
              a.ids[(int64_t)row * a.ldt] = a.id_map ? a.id_map[col] : col;
              if (a.prob) a.prob[(int64_t)row * a.ldt] = weight_float(mant, e) * zf;
            }
          }
        }
        return;
      }
      before += total;
    }
  }

  __device__ void write_probs(uint64_t tkey, float zf) {
    float* out = a.probs + (int64_t)row * a.ldp;
    const bool vec = (((uintptr_t)(out - off)) & 15) == 0;
    for (int v = vbeg + lane; v < vend; v += 32) {
      const uint4 r = get(v);
      float q[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float l = elem(r, j);
        const float ph = lead(l);
        q[j] = 0.0f;
        if (alive(ph) && at_least(l, v * VE + j - off, tkey)) {
          int e;
          const uint64_t mant = weight_mant(l, m, sc, ph, sh.tab, e);
          if (weight_fix(mant, e) >= minw) q[j] = weight_float(mant, e) * zf;
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
__global__ void __launch_bounds__(kT) sample_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char smem[];
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
  const char* l0 = (const char*)logits;
  const char* l1 = l0 + (((int64_t)rows - 1) * ld + n) * es;
  const char* p0 = (const char*)probs;
  if (probs && p0 < l1 && l0 < p0 + (((int64_t)rows - 1) * ldp + n) * 4) return TFD_ERR_INVALID;

  const int64_t nv = (n + ve - 1) / ve + 1;  // one more where a row starts off a 16-byte boundary
  const size_t fixed = (sizeof(Shared) + 15) / 16 * 16;
  const size_t room = 227 * 1024 - fixed;
  int dev = 0;
  const int sms = tfd_host::device_sms(dev);
  int c = 1;
  while (c < kMaxC && n / c > 2048 && ((int64_t)rows * c * 2 <= sms || nv / c * 16 > 100 * 1024))
    c *= 2;
  const size_t part = (size_t)((nv + c - 1) / c + 1) * 16;
  const bool keep = part <= room;
  const size_t smem = fixed + (keep ? part : 0);
  Args a = {logits, n, ld, temperature, top_k, top_p, min_p, u, id_map, ids, prob, ldt, probs, ldp,
            dev_status};
  cudaStream_t st = tfd_host::as_stream(stream);
#define TFD_SAMPLE_CASE(B, K) \
  if (bf16 == B && keep == K) \
    return tfd_host::launch_clusters<sample_kernel<B, K>>(a, rows, c, kT, smem, \
                                                          tfd_host::kSmemLimit, st);
  TFD_SAMPLE_CASE(true, true) TFD_SAMPLE_CASE(true, false)
  TFD_SAMPLE_CASE(false, true) TFD_SAMPLE_CASE(false, false)
#undef TFD_SAMPLE_CASE
  return TFD_ERR_UNSUPPORTED;
}
