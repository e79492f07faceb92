// paged_plan.cu - page tables and slot maps of a round from the requests' lengths, on the GPU.
//
// want_r = ceil((lens_r + n_r) / page_size); three prefix sums over the requests (rows, pages given
// back, pages missing) say where everything goes: page i given back (in the order of requests and
// pages) goes to free_ids[n_free + back - 1 - i], page i taken comes from free_ids[n_free + back - 1 -
// i], and row i of the round belongs to the request whose range of rows holds it. So every move and
// every row is found by a binary search of its own, whatever the requests' sizes.
//
// One cluster; every block forms the prefix sums for itself (12 bytes a request, from L2) and takes its
// share of the moves and rows, with a cluster barrier between pages given back, pages taken, and rows.
// Bound by latency: a few dependent reads and, when pages move, three barriers (4 requests 4.3 us, 2048 requests
// with 52000 rows 15.0).
#include <cooperative_groups.h>

#include "paged.cuh"

namespace {

using namespace tfd;
namespace cg = cooperative_groups;

constexpr int kBlocks = 8;  // blocks of the cluster where there is work for them

// A small round waits for barriers: with 256 threads it took 4.2 us, with 512 5.0. A large one has work for all (2048
// requests, 52000 rows: with 512 threads a block 14.8 us, with 1024 16.1). Both before ids that are no pages left the stack.
constexpr int threads_of(bool one) { return one ? 256 : 512; }

struct Args {
  const int32_t* lens;
  const int32_t* n_new;
  int32_t* table;
  int64_t ldt;
  int32_t* held;
  int32_t* free_ids;
  int32_t* n_free;
  int32_t* row_start;
  int32_t* slots;
  int32_t* pos;
  int32_t* dev_status;
  int64_t rows;
  int requests, page_size, max_pages, pages;
};

// Pages that lens + n tokens take (both >= 0).
__device__ __forceinline__ int64_t pages_of(int32_t len, int32_t n, int page_size) {
  const uint32_t t = (uint32_t)len + (uint32_t)n;
  return t ? (int64_t)((t - 1) / (uint32_t)page_size) + 1 : 0;
}

// The last r < n with first[r] <= i (first[0] = 0, not decreasing).
__device__ __forceinline__ int find(const int32_t* first, int n, int32_t i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int d) {
  const uint32_t lo = __shfl_up_sync(0xffffffffu, (uint32_t)v, d);
  const uint32_t hi = __shfl_up_sync(0xffffffffu, (uint32_t)((uint64_t)v >> 32), d);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Ids in free_ids[first .. end) that are no pages leave it, the others keep their order: a warp; where they end. A
// function of its own, as it is hardly ever called (its loop in the kernel: two plans of a large round 30.3 us, so 30.0).
__device__ __noinline__ int32_t without_none(int32_t* free_ids, int32_t first, int32_t end, int32_t pages) {
  const int lane = threadIdx.x & 31;
  int32_t to = first;
  for (int64_t i = first; i < end; i += 32) {
    const int32_t id = end - i > lane ? __ldcg(free_ids + i + lane) : -1;
    const bool in = id >= 0 && id < pages;
    const uint32_t ins = __ballot_sync(0xffffffffu, in);  // all 32 have been read
    if (in) free_ids[to + __popc(ins & ((1u << lane) - 1u))] = id;
    to += __popc(ins);
  }
  return to;
}

template <bool kOne>  // one block
__global__ void __launch_bounds__(threads_of(kOne)) page_plan_kernel(const Args a) {
  constexpr int kT = threads_of(kOne);
  extern __shared__ int32_t sm[];
  __shared__ int64_t warp_sums[3][kT / 32];
  __shared__ int32_t s_odd, s_top;  // a block of several met a page that is none; the lead's: the stack without them
  tfd_host::after_previous();
  cg::cluster_group cl = cg::this_cluster();
  const unsigned rank = kOne ? 0 : cl.block_rank(), blocks = kOne ? 1 : cl.num_blocks();
  auto sync = [&] {
    if (kOne) __syncthreads();
    else cl.sync();
  };
  const int R = a.requests, ps = a.page_size;
  int32_t* first[3] = {sm, sm + R + 1, sm + 2 * (R + 1)};  // rows, given back, missing
  uint8_t* bad = reinterpret_cast<uint8_t*>(sm + 3 * (R + 1));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_free = *a.n_free;
  const bool lead = rank == 0;
  if (!kOne && tid == 0) s_odd = 0;
  for (int r = tid; r < R; r += kT) {
    const int32_t len = a.lens[r], n = a.n_new[r], held = a.held[r];
    bool b = len < 0 || n < 0 || held < 0 || held > a.max_pages;
    int64_t want = held;
    if (!b) {
      want = pages_of(len, n, ps);
      b = want > a.max_pages || (uint32_t)len + (uint32_t)n > 0x7fffffffu;
      if (b) want = held;
    }
    if (b && lead) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
    first[0][r] = n > 0 ? n : 0;
    first[1][r] = held > want ? (int32_t)(held - want) : 0;
    first[2][r] = want > held ? (int32_t)(want - held) : 0;
    bad[r] = b;
  }
  __syncthreads();
  // exclusive prefix sums in place, a run of requests a thread; sums of rows past 2^31 - 1 stay there
  // (pages cannot: requests * max_pages is below)
  const int per = (R + kT - 1) / kT, r0 = min(R, tid * per), r1 = min(R, r0 + per);
  int64_t sum[3] = {0, 0, 0};
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    for (int r = r0; r < r1; ++r) sum[q] += first[q][r];
    int64_t x = sum[q];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = shfl_up64(x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[q][warp] = x;
    sum[q] = x - sum[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    int64_t at = sum[q], total = 0;
    for (int w = 0; w < kT / 32; ++w) {
      if (w < warp) at += warp_sums[q][w];
      total += warp_sums[q][w];
    }
    for (int r = r0; r < r1; ++r) {
      const int32_t n = first[q][r];
      first[q][r] = (int32_t)min(at, (int64_t)0x7fffffff);
      at += n;
    }
    if (tid == 0) first[q][R] = (int32_t)min(total, (int64_t)0x7fffffff);
  }
  __syncthreads();
  const int32_t back = first[1][R], missing = first[2][R];
  const bool broken = n_free < 0 || n_free > a.pages || (int64_t)n_free + back > a.pages;
  if (broken && lead && tid == 0) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
  int32_t top = broken ? 0 : n_free + back;
  // a request gets its pages if all that are missing up to it are there
  auto without = [&](int r) { return first[2][r + 1] > first[2][r] && first[2][r + 1] > top; };
  const int64_t t0 = (int64_t)rank * kT + tid, nt = (int64_t)blocks * kT;
  if (back > 0 || missing > 0) {
    bool odd = false;  // a page that is none is among those given back
    if (!broken) {
      for (int64_t i = t0; i < back; i += nt) {
        const int r = find(first[1], R, (int32_t)i);
        const int64_t at = pages_of(a.lens[r], a.n_new[r], ps) + (i - first[1][r]);
        const int32_t id = a.table[r * a.ldt + at];
        if (id < 0 || id >= a.pages) {
          set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
          odd = true;
        }
        a.free_ids[top - 1 - i] = id;
      }
    }
    // the stack is complete; every block has read what the requests held
    if (kOne) {
      odd = __syncthreads_or(odd);
    } else {
      if (odd) s_odd = 1;
      cl.sync();
      odd = back > 0 && __any_sync(0xffffffffu, lane < (int)blocks && *cl.map_shared_rank(&s_odd, lane));
    }
    if (odd) {
      // ids that are no pages leave the stack, or a sound request would get them; the others keep their order
      if (lead && warp == 0) {
        const int32_t to = without_none(a.free_ids, n_free, top, a.pages);
        if (lane == 0) s_top = to;
      }
      sync();
      top = kOne ? s_top : *cl.map_shared_rank(&s_top, 0);
    }
    for (int64_t i = t0; i < missing; i += nt) {
      const int r = find(first[2], R, (int32_t)i);
      const int64_t want = pages_of(a.lens[r], a.n_new[r], ps);
      const bool none = without(r);
      if (none) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
      // its missing pages end its table: the last is entry want - 1
      a.table[r * a.ldt + want - (first[2][r + 1] - i)] = none ? -1 : __ldcg(a.free_ids + (top - 1 - i));
    }
    for (int64_t r = t0; r < R; r += nt) {
      const bool moved = first[2][r + 1] > first[2][r] ? !without((int)r)
                                                       : !broken && first[1][r + 1] > first[1][r];
      if (moved) a.held[r] = (int32_t)pages_of(a.lens[r], a.n_new[r], ps);
    }
    if (t0 == 0 && !broken) {
      int lo = 0, hi = R + 1;  // the largest sum of missing pages that is there
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[2][mid] <= top) lo = mid;
        else hi = mid;
      }
      *a.n_free = top - first[2][lo];
    }
    sync();  // the tables are complete
  }
  for (int64_t r = t0; r <= R; r += nt) a.row_start[r] = first[0][r];
  const int32_t total = first[0][R];
  if (a.slots == nullptr) return;
  if (total > a.rows && t0 == 0) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
  // several rows a thread at once: each waits for a search and then for its page
  constexpr int kAtOnce = 4;
  for (int64_t i0 = t0; i0 < a.rows; i0 += kAtOnce * nt) {
    int32_t p[kAtOnce], pg[kAtOnce], id[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t i = i0 + u * nt;
      p[u] = id[u] = -1;
      if (i < total && i < a.rows) {
        const int r = find(first[0], R, (int32_t)i);
        if (!bad[r] && !without(r)) {
          p[u] = a.lens[r] + (int32_t)(i - first[0][r]);
          pg[u] = (int32_t)((uint32_t)p[u] / (uint32_t)ps);
          id[u] = __ldcg(a.table + r * a.ldt + pg[u]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t i = i0 + u * nt;
      if (i >= a.rows) break;
      int32_t slot = -1;
      if (p[u] >= 0) {
        if (id[u] >= 0 && id[u] < a.pages) slot = id[u] * ps + (p[u] - pg[u] * ps);
        else set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
      }
      a.slots[i] = slot;
      a.pos[i] = p[u];
    }
  }
}

}  // namespace

extern "C" tfd_status tfd_page_plan(const int32_t* lens, const int32_t* n_new, int requests,
                                    int page_size, int32_t* table, int64_t ldt, int max_pages,
                                    int32_t* held, int32_t* free_ids, int pages, int32_t* n_free,
                                    int32_t* row_start, int32_t* slots, int32_t* pos, int64_t rows,
                                    int32_t* dev_status, void* stream) {
  using tfd_host::aligned;
  if (!lens || !n_new || !table || !held || !free_ids || !n_free || !row_start)
    return TFD_ERR_INVALID;
  if ((slots == nullptr) != (pos == nullptr) || rows < 0 || (!slots && rows > 0))
    return TFD_ERR_INVALID;
  if (requests < 1 || page_size < 1 || page_size > TFD_MAX_PAGE || max_pages < 1 ||
      ldt < max_pages || pages < 1 || (int64_t)pages * page_size > 2147483647)
    return TFD_ERR_INVALID;
  if (requests > TFD_MAX_REQUESTS || rows > 2147483647 || ldt > ((int64_t)1 << 40) ||
      (int64_t)requests * max_pages > 2147483647)
    return TFD_ERR_UNSUPPORTED;
  const struct {
    const void* p;
    int64_t bytes;
  } all[] = {{lens, requests * 4ll},
             {n_new, requests * 4ll},
             {table, ((int64_t)(requests - 1) * ldt + max_pages) * 4},
             {held, requests * 4ll},
             {free_ids, pages * 4ll},
             {n_free, 4},
             {row_start, requests * 4ll + 4},
             {slots, rows * 4},
             {pos, rows * 4},
             {dev_status, 4}};
  const int count = sizeof(all) / sizeof(all[0]);
  for (int i = 0; i < count; ++i) {
    if (!aligned(all[i].p, 4)) return TFD_ERR_INVALID;
    for (int j = i < 2 ? 2 : i + 1; j < count; ++j)  // lens and n_new are only read
      if (tfd_host::overlap(all[i].p, all[i].bytes, all[j].p, all[j].bytes))
        return TFD_ERR_INVALID;
  }
  int dev = 0;
  tfd_host::device_sms(dev);
  const Args a = {lens,  n_new, table,      ldt,  held,     free_ids,  n_free,    row_start,
                  slots, pos,   dev_status, rows, requests, page_size, max_pages, pages};
  const size_t smem = (size_t)3 * 4 * (requests + 1) + requests;
  const int most = 3 * 4 * (TFD_MAX_REQUESTS + 1) + TFD_MAX_REQUESTS;
  // One block where that is at least as fast, by what the host knows: rows, or without them the pages that can move. One
  // block and eight, us, no page moved and pages taken and given back in turn: 4 requests x 6 rows 3.4 4.6 | 4.1 6.8;
  // 32 x 32 4.6 5.3 | 4.2 6.9; 128 x 8 5.1 5.7 | 4.4 6.9; 512 x 1 5.1 7.2 | 5.1 7.9; 1024 x 1 7.6 11.3 | 5.7 8.5;
  // 128 x 32 11.6 9.6 | 4.5 6.9; 512 x 8 13.6 12.3 | 4.8 7.8. Without rows, requests x pages each: 4 x 100 4.7 | 6.3;
  // 512 x 2 7.6 | 6.9; 32 x 100 11.1 | 6.7; 512 x 10 18.8 | 8.1; 512 x 1000 1423 | 104.
  const bool few = slots ? rows <= 1024 : (int64_t)requests * max_pages <= 2048;
  const int c = requests <= 512 && few ? 1 : kBlocks;
  cudaStream_t st = tfd_host::as_stream(stream);
  return c == 1
             ? tfd_host::launch_clusters<page_plan_kernel<true>>(a, dev, 1, 1, threads_of(true), smem, most, st)
             : tfd_host::launch_clusters<page_plan_kernel<false>>(a, dev, 1, c, threads_of(false), smem, most, st);
}
