// accept_sampled.cu - the rejection accept of sampled drafts, and the round's next token.
//
// Draft t of a stream is kept when all before it are and u_t q_t(d_t) < p_t(d_t): the product of two
// fp32 numbers is exact in 53 bits, so this decision has no rounding. The next token is drawn from
// max(p_m - q_m, 0) at the first draft turned down (from p_m where that is zero everywhere), or from
// p_m behind the last asked draft; kept drafts and next token are then distributed as if drawn from
// p one by one.
//
// The draw sums integers: each probability as a multiple of 2^-43 (weight.cuh gives the reasons),
// clamped to 0..1 with NaN as 0, so sums do not depend on the order and equal p and q leave exactly
// zero. One thread-block cluster takes a stream, every block decides its drafts for itself, each
// warp sums a contiguous part of the columns, and after one cluster barrier the block that holds
// the drawn column scans the part of the warp that holds it with all its threads.
//
// 4 x 5 x 163840 takes 7.5 us, all latency; 48 x 5 x 163840 17.6 us, 0.53 of the copy rate (one row
// of p and one of q a stream, 63 MB).
#include <cooperative_groups.h>

#include "launch.cuh"
#include "weight.cuh"

namespace {

using namespace tfd;
namespace cg = cooperative_groups;

constexpr int kT = 256;
constexpr int kW = kT / 32;
constexpr int kMaxC = tfd_host::kMaxCluster;
constexpr int kCols = 4;   // columns a lane takes at once
constexpr int kBatch = 4;  // such loads in flight

struct Args {
  const float* p;
  int64_t ldp;
  const float* q;
  int64_t ldq;
  int64_t n, nq;
  const int32_t* q_map;
  const int32_t* drafts;
  const int32_t* n_asked;
  const float* u;
  const float* u_next;
  int win;
  int32_t* n_kept;
  int32_t* next_ids;
  float* next_prob;
  unsigned long long* asked_hist;
  unsigned long long* kept_hist;
  int32_t* dev_status;
};

// max(p - q, 0) as an integer multiple of 2^-43, p and q clamped to 0..1 (NaN to 0). For p > q the
// difference is dh + dl exactly; it is cut into 21 bits and a signed rest below 2^-21, each taken
// from the low bits of a float to which 1.5 * 2^23 was added: no float-to-integer conversions,
// whose unit has a sixteenth of the FMA rate (48 x 163840 columns: 32.7 us with them).
__device__ __forceinline__ uint64_t rest_fix(float p, float q) {
  p = fminf(fmaxf(p, 0.0f), 1.0f);
  q = fminf(fmaxf(q, 0.0f), 1.0f);
  const float dh = fmaxf(__fsub_rn(p, q), 0.0f);
  const float dl = __fsub_rn(__fsub_rn(p, dh), q);
  const float magic = 12582912.0f;
  const float a = __fmaf_rn(dh, 2097152.0f, magic);
  const float top = __fsub_rn(a, magic);
  float rest = __fmaf_rn(dh, 2097152.0f, -top);              // exact, |rest| <= 1/2
  rest = __fmaf_rn(dl, 2097152.0f, rest);
  const float b = __fmaf_rn(rest, 4194304.0f, magic);
  const int64_t v = ((int64_t)(int32_t)(__float_as_uint(a) - 0x4B400000u) << 22) +
                    (int32_t)(__float_as_uint(b) - 0x4B400000u);
  return dh > 0.0f ? (uint64_t)v : 0;
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, (unsigned long long)v, m);
  return v;
}

struct Shared {
  uint64_t blocks[2][kMaxC];  // every block's mass of max(p - q, 0); of p, where that is zero
  uint64_t warps[kW];         // this block's warps'
  int fail, bad;
};

__global__ void __launch_bounds__(kT) accept_sampled_kernel(const Args a) {
  __shared__ Shared sh;
  tfd_host::after_previous();
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int s = blockIdx.x / C;
  const int na = a.n_asked[s];
  const bool counted = na >= 0 && na <= a.win;
  if (tid == 0) {
    sh.fail = counted ? na : 0;
    sh.bad = counted ? 0 : 1;
  }
  __syncthreads();
  const float* prow = a.p + (int64_t)s * (a.win + 1) * a.ldp;
  const float* qrow = a.q + (int64_t)s * a.win * a.ldq;
  const float un = a.u_next[s];
  if (counted) {
    for (int t = tid; t < na; t += kT) {
      const int d = a.drafts[(int64_t)s * a.win + t];
      const float ut = a.u[(int64_t)s * a.win + t];
      int dq = d;
      if (d < 0 || d >= a.n || !(ut >= 0.0f && ut < 1.0f)) {
        sh.bad = 1;
      } else {
        if (a.q_map) dq = a.q_map[d];
        const float qd = dq >= 0 && dq < a.nq ? qrow[(int64_t)t * a.ldq + dq] : 0.0f;
        const float pd = prow[(int64_t)t * a.ldp + d];
        if (!((double)ut * (double)qd < (double)pd)) atomicMin(&sh.fail, t);
      }
    }
  }
  if (tid == 0 && !(un >= 0.0f && un < 1.0f)) sh.bad = 1;
  __syncthreads();
  if (sh.bad) {  // the whole cluster sees the same
    if (rank == 0 && tid == 0) {
      a.n_kept[s] = 0;
      a.next_ids[s] = -1;
      if (a.next_prob) a.next_prob[s] = 0.0f;
      set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
    }
    return;
  }
  const int m = sh.fail;
  if (rank == 0) {
    if (tid == 0) a.n_kept[s] = m;
    if (a.asked_hist) {
      for (int i = tid; i < na; i += kT) atomicAdd(a.asked_hist + i, 1ull);
      for (int i = tid; i < m; i += kT) atomicAdd(a.kept_hist + i, 1ull);
    }
  }
  const bool rejected = m < na;
  prow += (int64_t)m * a.ldp;
  qrow += (int64_t)(rejected ? m : 0) * a.ldq;

  // columns in chunks of 128 a warp; each warp a contiguous range of chunks
  const int n = (int)a.n;
  const int off = (int)((uintptr_t)prow & 15) / 4;
  const int chunks = (off + n + 32 * kCols - 1) / (32 * kCols);
  const int per_c = (chunks + C - 1) / C, per_w = (per_c + kW - 1) / kW;
  const int cbeg = rank * per_c + warp * per_w;
  const int cend = min(min(cbeg + per_w, (rank + 1) * per_c), chunks);
  const bool qvec = !a.q_map && (((uintptr_t)(qrow - off)) & 15) == 0;

  bool from_p = !rejected;
  auto load = [&](int chunk, float4& p, float4& q) {
    const int c0 = chunk * 32 * kCols + lane * kCols - off;
    p = q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c0 >= 0 && c0 + kCols <= n) {
      p = __ldg((const float4*)(prow + c0));
      if (qvec && !from_p) q = __ldg((const float4*)(qrow + c0));
    } else {
      float* pv = &p.x;
      float* qv = &q.x;
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const int c = c0 + j;
        if (c < 0 || c >= n) continue;
        pv[j] = prow[c];
        if (qvec && !from_p) qv[j] = qrow[c];
      }
    }
    if (!qvec && !from_p) {
      float* qv = &q.x;
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const int c = c0 + j;
        if (c < 0 || c >= n) continue;
        const int k = a.q_map ? a.q_map[c] : c;
        if (k >= 0 && k < a.nq) qv[j] = qrow[k];
      }
    }
  };

  // the masses; a second round over p alone where nothing of it lies above q
  uint64_t total = 0;
  const uint64_t* blocks = sh.blocks[0];
  for (int round = 0; round < 2; ++round) {
    uint64_t sum = 0;
    for (int c = cbeg; c < cend; c += kBatch) {
      float4 p[kBatch], q[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        p[i] = q[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c + i < cend) load(c + i, p[i], q[i]);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        sum += rest_fix(p[i].x, q[i].x) + rest_fix(p[i].y, q[i].y) + rest_fix(p[i].z, q[i].z) +
               rest_fix(p[i].w, q[i].w);
    }
    sum = warp_sum64(sum);
    if (lane == 0) sh.warps[warp] = sum;
    if (round == 0) cl.sync();  // every block runs, and this block's sums are written
    else __syncthreads();
    if (tid < C) {
      uint64_t x = 0;
      for (int w = 0; w < kW; ++w) x += sh.warps[w];
      *cl.map_shared_rank(&sh.blocks[round][rank], tid) = x;
    }
    cl.sync();
    blocks = sh.blocks[round];
    for (int c = 0; c < C; ++c) total += blocks[c];
    if (total != 0 || from_p) break;
    from_p = true;
  }
  if (total == 0) {
    if (rank == 0 && tid == 0) {
      a.next_ids[s] = -1;
      if (a.next_prob) a.next_prob[s] = 0.0f;
    }
    return;
  }
  const uint64_t target = mul_frac(un, total, false);
  uint64_t before = 0;
  for (int c = 0; c < rank; ++c) before += blocks[c];
  if (target < before || target >= before + blocks[rank]) return;
  // The warp whose columns hold the target, then those columns by the whole block, a chunk a warp.
  uint64_t ws = lane < kW ? sh.warps[lane] : 0, incl = ws;
#pragma unroll
  for (int o = 1; o < kW; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, (unsigned long long)incl, o);
    if (lane >= o) incl += x;
  }
  const int at = __ffs(__ballot_sync(0xffffffffu, before + incl > target)) - 1;
  before += __shfl_sync(0xffffffffu, (unsigned long long)(incl - ws), at);
  const int c0 = rank * per_c + at * per_w;
  const int c1 = min(min(c0 + per_w, (rank + 1) * per_c), chunks);
#pragma unroll 1
  for (int c = c0 + warp; c - warp < c1; c += kW) {
    float4 p, q;
    p = q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < c1) load(c, p, q);
    const uint64_t r[kCols] = {rest_fix(p.x, q.x), rest_fix(p.y, q.y), rest_fix(p.z, q.z),
                               rest_fix(p.w, q.w)};
    const uint64_t sum = r[0] + r[1] + r[2] + r[3];
    incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t x = __shfl_up_sync(0xffffffffu, (unsigned long long)incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) sh.warps[warp] = incl;
    __syncthreads();
    const uint64_t mine = lane < kW ? sh.warps[lane] : 0;
    uint64_t run = before + warp_sum64(lane < warp ? mine : 0) + incl - sum;
    before += warp_sum64(mine);
    if (run <= target && run + sum > target) {
      bool done = false;
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        run += r[j];
        if (!done && run > target) {
          done = true;
          a.next_ids[s] = c * 32 * kCols + lane * kCols - off + j;
          if (a.next_prob) a.next_prob[s] = __ull2float_rn(r[j]) / __ull2float_rn(total);
        }
      }
    }
    if (before > target) return;
  }
}

}  // namespace

extern "C" tfd_status tfd_accept_sampled(const float* p, int64_t ldp, const float* q, int64_t ldq,
                                         int64_t n, int64_t nq, const int32_t* q_map,
                                         const int32_t* drafts, const int32_t* n_asked,
                                         const float* u, const float* u_next, int streams, int win,
                                         int32_t* n_kept, int32_t* next_ids, float* next_prob,
                                         int64_t* asked_hist, int64_t* kept_hist,
                                         int32_t* dev_status, void* stream) {
  using tfd_host::aligned;
  if (!p || !q || !drafts || !n_asked || !u || !u_next || !n_kept || !next_ids)
    return TFD_ERR_INVALID;
  if (streams < 1 || win < 1 || win > TFD_MAX_TOPK || n < 1 || nq < 1 || ldp < n || ldq < nq)
    return TFD_ERR_INVALID;
  if (!q_map && nq != n) return TFD_ERR_INVALID;
  if ((asked_hist == nullptr) != (kept_hist == nullptr)) return TFD_ERR_INVALID;
  if (n > kMaxDrawCols || nq > kMaxDrawCols || streams > (1 << 24)) return TFD_ERR_UNSUPPORTED;
  if (!aligned(p, 4) || !aligned(q, 4)) return TFD_ERR_INVALID;
  for (const void* x : {(const void*)q_map, (const void*)drafts, (const void*)n_asked,
                        (const void*)u, (const void*)u_next, (const void*)n_kept,
                        (const void*)next_ids, (const void*)next_prob, (const void*)dev_status})
    if (x && !aligned(x, 4)) return TFD_ERR_INVALID;
  if (asked_hist && (!aligned(asked_hist, 8) || !aligned(kept_hist, 8))) return TFD_ERR_INVALID;
  // outputs apart from the inputs: a stream's blocks read them for themselves
  const int64_t four = (int64_t)streams * 4;
  const struct { const void* p; int64_t bytes; } outs[] = {
      {n_kept, four}, {next_ids, four}, {next_prob, four}, {asked_hist, (int64_t)win * 8},
      {kept_hist, (int64_t)win * 8}},
      ins[] = {{p, (((int64_t)streams * (win + 1) - 1) * ldp + n) * 4},
               {q, (((int64_t)streams * win - 1) * ldq + nq) * 4}, {q_map, n * 4},
               {drafts, four * win}, {n_asked, four}, {u, four * win}, {u_next, four}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (tfd_host::overlap(o.p, o.bytes, i.p, i.bytes)) return TFD_ERR_INVALID;
  // blocks a stream: the fewest rounds of what the device holds at once, each costing about as much
  // as 4096 columns besides its blocks' own
  int dev = 0;
  tfd_host::device_sms(dev);
  if (!tfd_host::allow_clusters<accept_sampled_kernel>(dev, 0)) return TFD_ERR_CUDA;
  const int c = tfd_host::cheapest_cluster(
      streams,
      [&](int i) { return tfd_host::clusters_at_once<accept_sampled_kernel>(dev, i, kT, 0); },
      [](int) { return true; },
      [&](int i, int64_t rounds) { return rounds * (4096 + 64 * i + n / i); });
  if (c == 0) return TFD_ERR_UNSUPPORTED;
  Args a = {p, ldp, q, ldq, n, nq, q_map, drafts, n_asked, u, u_next, win, n_kept, next_ids,
            next_prob, reinterpret_cast<unsigned long long*>(asked_hist),
            reinterpret_cast<unsigned long long*>(kept_hist), dev_status};
  return tfd_host::launch_clusters<accept_sampled_kernel>(a, dev, streams, c, kT, 0, 0,
                                                          tfd_host::as_stream(stream));
}
