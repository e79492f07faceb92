// lora_tc.cu - low-rank adapters over prompts: y_r = base_r + s_a B_a (A_a x_r) for tiles of 128 rows of
// one adapter, on the tensor cores with their accumulators in tensor memory.
//
// A 4096-wide projection of a 128-row tile reads 1 MB of x, 1 MB of base, writes 1 MB of y and, at rank
// 64, takes 1 MB of the adapter from L2: enough rows a tile keep the adapter's share small (at 32
// rows it was twice all the rest), and at that size warp-level MMAs would bound it (21 us of 12.9
// GFLOP for 4099 rows at rank 64, against 16 us for the bytes); tcgen05.mma does not.
//
// A thread-block cluster takes a tile. Shrink: D1 = x A^T (128 rows x rank), the k range split over the
// cluster's blocks; x rows (gathered by index) and A come through a ring of shared-memory stages of
// 64 k by asynchronous 16-byte copies, placed in the 128-byte swizzle that the matrix descriptors
// name. The blocks' partial sums are added in block order through distributed shared memory, scaled,
// and split into bf16 parts that add up to them (two where y is bf16: 2^-17 relative, under its 2^-9
// rounding; three, all 24 bits, where it is fp32). Expand: D2 = h B^T in chunks of outputs that are
// 128 bytes of a row of y, the parts' products added in the same fp32 accumulators; a chunk's B and base
// rows are copied ahead, its products run while the chunk before it is written, its base takes the
// sums and is written out from shared memory in whole 128-byte rows.
//
// Measured, 4096 to 4096 in bf16: 4099 rows of six adapters at rank 64 in 44.1 us, 0.36 of the copy
// rate (62.7 with the sums read by every block, 54.4 with a chunk's products waited for); 16384 rows 148
// us, 0.40; 32768 rows 264 us, 0.45. Bound by the latency of the copies in flight, not by the MMAs.
#include <cooperative_groups.h>

#include "lora.cuh"

namespace {

using namespace tfd;
using namespace tfd_adapters;
namespace cg = cooperative_groups;

constexpr int kNT = 512;           // threads
constexpr int kRows = 128 * 8 / kNT;  // rows of a 128-byte-wide tile that a thread copies 16 bytes of
constexpr int kTM = 128;           // rows of a tile: tensor-memory lanes
constexpr int kKB = 64;            // k of a stage: 128 bytes of a row
constexpr int kXBytes = kTM * 128;  // x of a stage; a chunk of base rows; h's 64 ranks of one part
constexpr int kStages = 4;
constexpr int kTmemCols = 256;     // D1 in the first 128, two D2 buffers of 64 behind it

__device__ __forceinline__ uint32_t sa(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// What threads wrote to shared memory becomes visible to the tensor cores' reads.
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void bar_init(uint32_t bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
}
// Bounded wait for the phase of parity `par` (about a second of global time); false on timeout.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t par) {
  uint64_t t0 = 0;
  for (int it = 0;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(par)
        : "memory");
    if (ok) return true;
    uint64_t now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
    if (it == 0) t0 = now;
    else if (now - t0 > 1000000000ull) return false;
  }
}
// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Instruction descriptor of kind::f16: fp32 accumulator, bf16 operands, both K-major, 128 x n.
__device__ __forceinline__ uint32_t idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kTM >> 4) << 24);
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
// 16 consecutive accumulator columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 8 of them.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Shared memory. The shrink's stages take all of it; then come the blocks' sums, the h parts and the
// expand's chunks. The sums lie where h comes later if the rank is at most 64, so that a thread can
// hold its share of h in between, and else where the chunks come later.
struct Layout {
  int r16;         // rank rounded up to 16
  int atoms;       // 64-rank pieces of h and B
  int parts;       // bf16 parts of h
  int cols;        // outputs of a chunk
  uint32_t h, sums, bufs, bars;  // offsets
  uint32_t stage;  // bytes of a stage
  uint32_t chunk;  // bytes of a chunk's B
  uint32_t bytes;
};
__host__ __device__ inline Layout layout(int rank, bool f32, int bufs) {
  Layout l;
  l.r16 = (rank + 15) / 16 * 16;
  l.atoms = (rank + 63) / 64;
  l.parts = f32 ? 3 : 2;
  l.cols = f32 ? 32 : 64;
  const uint32_t h = (uint32_t)(l.parts * l.atoms * kXBytes);
  const uint32_t sums = ((uint32_t)(kTM * (l.r16 + 4) * 4) + 1023) / 1024 * 1024;
  l.h = 0;
  l.sums = l.atoms == 1 ? 0 : h;
  l.bufs = l.atoms == 1 && sums > h ? sums : h;
  l.stage = kXBytes + (uint32_t)l.r16 * 128;
  l.chunk = (uint32_t)(l.atoms * l.cols * 128);
  const uint32_t shrink = kStages * l.stage, expand = l.bufs + bufs * (l.chunk + kXBytes);
  l.bars = shrink > expand ? shrink : expand;
  if (l.bars < l.sums + sums) l.bars = l.sums + sums;
  l.bytes = l.bars + 128;
  return l;
}

// kBufs: chunks of the expand in shared memory.
template <int kBufs>
__global__ void __launch_bounds__(kNT, 2) lora_tc_kernel(const Args a) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ int32_t tile_rows[kTM];
  tfd_host::after_previous();
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank_c = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Layout l = layout(a.rank, a.f32, kBufs);
  int key = 0;
  const int m =
      find_tile<kTM, kNT>(a, blockIdx.x / C, tile_rows, reinterpret_cast<int32_t*>(smem), key);
  if (m == 0) return;  // all blocks of the cluster alike
  const bool none = key == a.n_adapters;
  if (none && a.base == a.y) return;
  __syncthreads();  // the counts are done with

  const int es = a.f32 ? 4 : 2, per = 16 / es;  // outputs in 16 bytes
  const int chunks = (a.n + l.cols - 1) / l.cols;
  const int j0 = (int)((int64_t)chunks * rank_c / C), j1 = (int)((int64_t)chunks * (rank_c + 1) / C);
  // a thread copies 16 bytes of kRows rows, 64 apart: piece tid % 8 of each
  const int piece = tid & 7, row0 = tid >> 3;

  if (none) {  // y = base, or zeros
    for (int j = j0; j < j1; ++j)
      for (int i = 0; i < kRows; ++i) {
        const int row = row0 + 64 * i, o = j * l.cols + piece * per;
        if (row >= m || o >= a.n) continue;
        const char* b = a.base ? a.base + (tile_rows[row] * a.ldb + o) * es : nullptr;
        char* y = a.y + (tile_rows[row] * a.ldy + o) * es;
        if (o + per <= a.n) {
          *reinterpret_cast<uint4*>(y) =
              b ? *reinterpret_cast<const uint4*>(b) : make_uint4(0u, 0u, 0u, 0u);
        } else {
          for (int e = 0; e < (a.n - o) * es; ++e) y[e] = b ? b[e] : 0;
        }
      }
    return;
  }

  const uint32_t s_h = sa(smem + l.h), s_ring = sa(smem), s_bufs = sa(smem + l.bufs), bars = sa(smem + l.bars);
  auto empty = [&](int s) { return bars + 8u * s; };              // stage s has been read
  const uint32_t shrunk = bars + 8u * kStages;                    // D1 is complete
  auto done = [&](int b) { return bars + 8u * (kStages + 1 + b); };  // D2 buffer b is complete
  const uint32_t drained = bars + 8u * (kStages + 3);  // every product is, after a wait ran out
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + l.bars + 64);
  if (tid == 0) {
    for (int s = 0; s < kStages + 4; ++s) bar_init(bars + 8u * s);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     sa(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;  // none of this thread's waits has run out; thread 0 issues products only so long

  // ---- shrink -----------------------------------------------------------------------------------
  const int kblocks = (a.k + kKB - 1) / kKB;
  const int k0 = (int)((int64_t)kblocks * rank_c / C), k1 = (int)((int64_t)kblocks * (rank_c + 1) / C);
  const int nk = k1 - k0;
  const __nv_bfloat16* xr[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)  // rows past the tile's last repeat it; their sums are not used
    xr[i] = a.x + (int64_t)tile_rows[min(row0 + 64 * i, m - 1)] * a.ldx + piece * 8;
  const __nv_bfloat16* aw = a.a + ((int64_t)key * a.rank + row0) * a.k + piece * 8;
  auto swz = [&](int row) { return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4)); };
  auto load_stage = [&](int i) {
    if (i < nk) {
      const uint32_t st = s_ring + (uint32_t)(i % kStages) * l.stage;
      const int kk = (k0 + i) * kKB;
      const uint32_t bytes = kk + piece * 8 < a.k ? 16u : 0u;
#pragma unroll
      for (int q = 0; q < kRows; ++q)
        copy16(st + swz(row0 + 64 * q), bytes ? (const void*)(xr[q] + kk) : (const void*)a.x, bytes);
      for (int row = row0; row < l.r16; row += 64) {
        const uint32_t in = row < a.rank ? bytes : 0u;
        copy16(st + kXBytes + swz(row),
               in ? (const void*)(aw + (int64_t)(row - row0) * a.k + kk) : (const void*)a.a, in);
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load_stage(i);
  const uint32_t desc1 = idesc(l.r16);
  for (int i = 0; i < nk; ++i) {
    copy_wait<kStages - 2>();
    fence_async();
    __syncthreads();
    if (tid == 0 && ok) {
      fence_after();
      const uint32_t st = s_ring + (uint32_t)(i % kStages) * l.stage;
      const uint64_t da = sdesc(st), db = sdesc(st + kXBytes);
#pragma unroll
      for (int kk = 0; kk < kKB / 16; ++kk) mma(tmem, da + 2u * kk, db + 2u * kk, desc1, (i | kk) != 0);
      mma_commit(empty(i % kStages));
    }
    if (i >= 1 && i + kStages - 1 < nk && ok)  // the stage to fill next was read by step i - 1
      ok = bar_wait(empty((i - 1) % kStages), (uint32_t)((i - 1) / kStages) & 1u);
    load_stage(i + kStages - 1);
  }
  if (nk > 0) {
    if (tid == 0 && !TFD_TEST_STALL_EXCHANGE) mma_commit(shrunk);
    if (ok) ok = bar_wait(shrunk, 0);
  }
  copy_wait<0>();
  fence_after();
  __syncthreads();

  auto b_of = [&](int buf) { return l.bufs + (uint32_t)buf * (l.chunk + kXBytes); };
  // this thread's 16-byte pieces of a chunk's B (rows of r16 ranks), and of its rows of base and y
  const int b_pieces = l.r16 / 8;
  const __nv_bfloat16* b_from[2];
  uint32_t b_to[2];
  int b_row[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {  // at most 64 rows of 16 pieces
    const int i = tid + q * kNT, row = i / b_pieces, p = i % b_pieces;
    b_row[q] = p * 8 < a.rank ? row : a.n;  // ranks past the adapter's: zeros
    if (row >= l.cols) b_row[q] = -1;
    b_from[q] = a.b + ((int64_t)key * a.n + row) * a.rank + p * 8;
    b_to[q] = (uint32_t)((p / 8) * l.cols * 128 + row * 128 + (((p % 8) ^ (row & 7)) << 4));
  }
  int64_t row_of[kRows];
#pragma unroll
  for (int q = 0; q < kRows; ++q) row_of[q] = row0 + 64 * q < m ? tile_rows[row0 + 64 * q] : -1;
  auto load_chunk = [&](int j) {
    if (j < j1) {
      const uint32_t st = s_bufs + (uint32_t)((j - j0) % kBufs) * (l.chunk + kXBytes);
      const int o0 = j * l.cols;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (b_row[q] >= 0) {
          const bool in = o0 + b_row[q] < a.n;
          copy16(st + b_to[q], in ? (const void*)(b_from[q] + (int64_t)o0 * a.rank) : (const void*)a.b,
                 in ? 16u : 0u);
        }
      if (a.base) {
        const int o = o0 + piece * per, left = (a.n - o) * es;
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
          const uint32_t bytes = row_of[q] >= 0 && left > 0 ? (uint32_t)min(left, 16) : 0u;
          copy16(st + l.chunk + swz(row0 + 64 * q),
                 bytes ? (const void*)(a.base + (row_of[q] * a.ldb + o) * es) : (const void*)a.base,
                 bytes);
        }
      }
    }
    copy_commit();
  };
  auto first_chunks = [&]() {
#pragma unroll
    for (int i = 0; i < kBufs - 1; ++i) load_chunk(j0 + i);
  };
  if (l.atoms == 1) first_chunks();  // on their way while h is summed

  // this block's sums, a row a thread
  const int rp = l.r16 + 4;  // floats of a row: 16-byte pieces of 8 rows in different banks
  float* sums = reinterpret_cast<float*>(smem + l.sums);
  for (int c = 16 * (warp >> 2); c < l.r16; c += 64) {  // four warps a quarter of the rows
    const int row = 32 * (warp & 3) + lane;
    float v[16];
    tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)c, v);
#pragma unroll
    for (int e = 0; e < 16; e += 4)
      *reinterpret_cast<float4*>(sums + row * rp + c + e) =
          nk > 0 ? make_float4(v[e], v[e + 1], v[e + 2], v[e + 3])
                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  fence_before();
  cl.sync();
  // All blocks' sums in order, scaled: each block takes its share of the tile, 8 ranks of a row at a
  // time, and brings every block the parts of h (reading all of the others' sums took 7 us at rank
  // 64 and four blocks).
  const float scale = a.scales ? a.scales[key] : 1.0f;
  const int pieces8 = l.r16 / 8, items = kTM * pieces8;
  const int i0 = items * rank_c / C, i1 = items * (rank_c + 1) / C;
  auto sum_of = [&](int i, float (&v)[8]) {
    const int at = i / pieces8 * rp + i % pieces8 * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll 4
    for (int r = 0; r < C; ++r) {
      const float4* p = reinterpret_cast<const float4*>(cl.map_shared_rank(sums, r) + at);
      const float4 x = p[0], y = p[1];
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
      v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
    }
    const bool in = i % pieces8 * 8 < a.rank;  // past the adapter's ranks 0 x inf would be NaN
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = in ? v[e] * scale : 0.0f;
  };
  auto put_h = [&](int i, float (&v)[8]) {
    const int row = i / pieces8, c = i % pieces8 * 8;
    for (int part = 0; part < l.parts; ++part) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat16 x = take_part(v[2 * e]), y = take_part(v[2 * e + 1]);
        w[e] = (uint32_t)__bfloat16_as_ushort(x) | ((uint32_t)__bfloat16_as_ushort(y) << 16);
      }
      unsigned char* at = smem + l.h + (part * l.atoms + c / 64) * kXBytes + row * 128 +
                          (((c % 64 / 8) ^ (row & 7)) << 4);
      for (int r = 0; r < C; ++r)
        *reinterpret_cast<uint4*>(cl.map_shared_rank(at, r)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };
  if (l.atoms == 1) {
    float v[kRows][8];  // at most 8 items a row
#pragma unroll
    for (int q = 0; q < kRows; ++q)
      if (i0 + tid + q * kNT < i1) sum_of(i0 + tid + q * kNT, v[q]);
    cl.sync();  // every block has read all sums: h takes their place
#pragma unroll
    for (int q = 0; q < kRows; ++q)
      if (i0 + tid + q * kNT < i1) put_h(i0 + tid + q * kNT, v[q]);
  } else {
    for (int i = i0 + tid; i < i1; i += kNT) {
      float v[8];
      sum_of(i, v);
      put_h(i, v);
    }
  }
  asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");  // for the MMAs that read h
  cl.sync();  // h is here, and no block reads or writes another's memory from now on
  if (l.atoms > 1) first_chunks();

  // ---- expand -----------------------------------------------------------------------------------
  // The products of a chunk run while the one before it is added to its base and written.
  const uint32_t desc2 = idesc(l.cols);
  auto multiply = [&](int i) {
    fence_after();
    const uint32_t st = s_bufs + (uint32_t)(i % kBufs) * (l.chunk + kXBytes);
    const uint32_t acc = tmem + 128u + (uint32_t)((i & 1) * 64);
    bool more = false;
    const uint64_t dh = sdesc(s_h), db = sdesc(st);  // advanced by units of 16 bytes
    for (int part = 0; part < l.parts; ++part)
      for (int kk = 0; kk < l.r16 / 16; ++kk) {
        mma(acc, dh + (uint32_t)((part * l.atoms + (kk >> 2)) * (kXBytes / 16) + 2 * (kk & 3)),
            db + (uint32_t)((kk >> 2) * l.cols * 8 + 2 * (kk & 3)), desc2, more);
        more = true;
      }
    mma_commit(done(i & 1));
  };
  copy_wait<kBufs - 2>();
  fence_async();
  __syncthreads();
  if (tid == 0 && ok && j0 < j1) multiply(0);
  for (int j = j0; j < j1; ++j) {
    const int i = j - j0, buf = i % kBufs, d = i & 1;
    copy_wait<kBufs - 3>();
    fence_async();
    __syncthreads();  // the next chunk is here; the last one's rows have been written from its buffer
    if (tid == 0 && ok && j + 1 < j1) multiply(i + 1);
    load_chunk(j + kBufs - 1);  // into the buffer of the chunk before this one
    if (ok) ok = bar_wait(done(d), (uint32_t)(i >> 1) & 1u);
    fence_after();
    // four warps a quarter of the rows, a quarter of a row a thread: two pieces of the base, in place
    const int row = 32 * (warp & 3) + lane, w4 = warp >> 2;
    const uint32_t acc = tmem + 128u + (uint32_t)(d * 64 + w4 * (l.cols / 4)) +
                         ((uint32_t)(32 * (warp & 3)) << 16);
    unsigned char* rows = smem + b_of(buf) + l.chunk + row * 128;
    uint4* p0 = reinterpret_cast<uint4*>(rows + (((2 * w4) ^ (row & 7)) << 4));
    uint4* p1 = reinterpret_cast<uint4*>(rows + (((2 * w4 + 1) ^ (row & 7)) << 4));
    uint4 x[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (a.base) {
      x[0] = *p0;
      x[1] = *p1;
    }
    float v[16];
    if (a.f32) {
      tmem_ld8(acc, v);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        x[c].x = __float_as_uint(__uint_as_float(x[c].x) + v[4 * c]);
        x[c].y = __float_as_uint(__uint_as_float(x[c].y) + v[4 * c + 1]);
        x[c].z = __float_as_uint(__uint_as_float(x[c].z) + v[4 * c + 2]);
        x[c].w = __float_as_uint(__uint_as_float(x[c].w) + v[4 * c + 3]);
      }
    } else {
      tmem_ld16(acc, v);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t* w = &x[c].x;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = (uint32_t)f32_to_bf16_bits(bf16_lo(w[e]) + v[8 * c + 2 * e]) |
                 ((uint32_t)f32_to_bf16_bits(bf16_hi(w[e]) + v[8 * c + 2 * e + 1]) << 16);
      }
    }
    *p0 = x[0];
    *p1 = x[1];
    fence_before();
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const int o = j * l.cols + piece * per;
      if (row_of[q] < 0 || o >= a.n) continue;
      const uint4 x = *reinterpret_cast<const uint4*>(smem + b_of(buf) + l.chunk + swz(row0 + 64 * q));
      char* y = a.y + (row_of[q] * a.ldy + o) * es;
      if (o + per <= a.n) {
        *reinterpret_cast<uint4*>(y) = x;
      } else if (a.f32) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (o + e < a.n) reinterpret_cast<uint32_t*>(y)[e] = w[e];
      } else {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (o + e < a.n) reinterpret_cast<uint16_t*>(y)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
  copy_wait<0>();
  if (!ok) {
    set_dev_status(a.dev_status, TFD_ERR_TIMEOUT);
    // no product may still read or write when this block's memory is given back (where no wait of
    // thread 0 ran out, it has waited for the last of them)
    if (tid == 0) {
      mma_commit(drained);
      bar_wait(drained, 0);
    }
  }
  __syncthreads();
  if (warp == 0) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
  }
}

}  // namespace

namespace {

// An adapter's last tile is half full if nothing is known of the ids.
int64_t likely_tiles(const Args& a) { return (a.rows + a.n_adapters * (kTM / 2) + kTM - 1) / kTM; }

template <int kBufs>
tfd_status launch(Args a, int dev, cudaStream_t stream, bool* taken) {
  const Layout l = layout(a.rank, a.f32, kBufs);
  size_t smem = l.bytes + 1024;
  const size_t counts = (size_t)4 * (a.n_adapters + 1) + 1024;
  if (smem < counts) smem = counts;
  const int most = 226 * 1024;  // with the static part: 227 KB
  a.smem = (int)smem - 1024;
  if (smem > (size_t)most || !tfd_host::allow_clusters<lora_tc_kernel<kBufs>>(dev, most))
    return TFD_OK;
  // Blocks a tile: as many as give every block an SM of its own (two on one slow each other down
  // here, 4099 rows at rank 64: 4 blocks 48 us, 7 84), within one round of clusters.
  const int64_t likely = likely_tiles(a);
  const int64_t tiles = (int64_t)a.rows / kTM + a.n_adapters + 1;
  const int sms = tfd_host::device_sms(dev);
  int c = 1;
  while (c < 8 && likely * (c + 1) <= sms &&
         likely <= (smem <= 112 * 1024  // two blocks an SM, or one
                        ? tfd_host::clusters_at_once<lora_tc_kernel<kBufs>, 0>(dev, c + 1, kNT, smem)
                        : tfd_host::clusters_at_once<lora_tc_kernel<kBufs>, 1>(dev, c + 1, kNT, smem)))
    ++c;
  *taken = true;
  return tfd_host::launch_clusters<lora_tc_kernel<kBufs>>(a, dev, tiles, c, kNT, smem, most, stream);
}

}  // namespace

tfd_status tfd_adapters::launch_tc(Args a, int dev, cudaStream_t stream, bool* taken) {
  *taken = false;
  const int each = (a.rows + a.n_adapters - 1) / a.n_adapters;
  if (!a.vec || each < 96 || a.rows <= kSmallRows || a.k < kKB) return TFD_OK;
  // Three chunks let two blocks share an SM, which pays once there are more tiles than SMs (32768 rows
  // at rank 64: 264 us, with four 328); a block alone hides more behind four (16384 rows: 147 and 156).
  if (likely_tiles(a) > tfd_host::device_sms(dev)) return launch<3>(a, dev, stream, taken);
  return launch<4>(a, dev, stream, taken);
}
