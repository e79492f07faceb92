// paged_attn.cu - attention of a request's new rows over its tokens in a paged key-value cache, on the
// tensor cores with accumulators in tensor memory: one pass with a running sum against a reference near
// the running maximum, split over the cache's length and joined.
//
// Work. A unit is one request, one key head, and up to N = 16, 32 or 64 of its (row, query head) pairs, which
// share every key and value read. The units' tokens, cut into tiles of 128, form one line over all requests;
// each block takes an equal stretch of it, found by a prefix sum over the requests that every block forms
// for itself, so lengths can stay on the GPU and long requests spread over all SMs. A stretch that
// covers a unit writes its rows; the others leave (reference, sum, weighted values) in the workspace, and
// the block that arrives last adds the unit's pieces in their order along the line (a counter for each block
// in which a unit begins; nobody waits for another block, and the sums' order does not depend on who is last).
//
// A tile: S^T = K q'^T (128 tokens x N) and O^T += V^T P^T (dim x N). With the tokens and the dims as the 128
// rows of the products no part of them is padding however few rows there are, and keys and values are read
// from shared memory as they come: keys as rows of dims, values as columns (MN-major). Both products read the
// cache's operand once: q' and the weights are two bf16 numbers a value (2^-16), side by side as columns, which
// costs next to nothing here (N of 64 columns takes the time of reading the 128 rows). E4M3 keys and values are
// multiplied as they are (kind::f8f6f4, against bf16 there is no product): q' over a power of two as four E4M3
// parts (2^-16), the weights as f16 cut into four E5M2 parts (an E5M2 number is the upper byte of an f16
// one), the last two parts of each times 2^8. An E4M3 value's scale is a summand of the score that its weight
// comes from, so weights stay in range; the sum, in which it is not, for scales up to 2^80.
//
// Roles. Two warps fetch (cp.async, 16 bytes a lane, up to 192 KB ahead), one thread finds the pieces and
// issues the scores' products, one the values'; the rest are softmax groups of 128 threads, a token each,
// 16 rows a group, later a dim each. At 16 rows two groups take tiles in turn (bf16, 128 dims), or two blocks
// share an SM (E4M3; 64 dims): a tile's chain of waits is longer than its bytes take. A weight may pass its
// reference by 2^8 (E4M3: 2^7) before the reference and the sums move, so after a piece's first tile they hardly do.
//
// What a row does not see gets a score of -inf and a weight of zero; tokens past the last and on bad pages are
// zero-filled. Zero times an infinity or NaN would be NaN: bf16 values that are not finite, of tokens that not
// all rows see, leave the product and are added at the end to the rows that see them.
//
// Measured: 96 requests of 1000 to 16000 tokens, 4 rows, 32/8 heads of 128 in bf16 493 us, 0.99 of the copy
// rate (3.3 GB); one row over 131041 tokens 95 (0.83); 24 verify windows of up to 6 rows 69 (0.72); 64 E4M3
// requests of 300 to 9000 tokens 130 (0.72); one draft step of four streams 17. Short pieces are bound by
// what beginning and ending one takes (about 8 us of chained waits, much of it instructions fetched for the
// first time), which the line's cuts allow for; kernels on warp-level products, two blocks an SM, measured
// 569, 112, 142, 208 and 22. Fetching by tensor maps (one warp, boxes of a page) measured no faster.
#include <cuda_fp16.h>

#include "paged.cuh"

namespace {

using namespace tfd;

constexpr int kTile = 128;                   // tokens of a tile
constexpr int kCols = 16;                    // rows of a unit that one softmax group takes
constexpr int kGroup = 128;                  // its threads, one a token; then one a dim
constexpr int kAhead = 3;                    // pieces found ahead
// A unit's end keeps its last kKeep tiles, and a unit of fewer than kLeast is not cut: a piece that small costs more,
// being joined, than it takes off its neighbour (four streams of 5 tiles a head 16.9 us, cut 23.8; verify windows 69.1,
// with ends of 3 tiles 71.6, units of fewer than 12 whole 71.7).
constexpr int kKeep = 1, kLeast = 6;
// Places on the line that beginning a unit takes, in tiles of its type: its query, its first and last tiles and its
// sums cost a block about that. The blocks' times even out by it (in turn on one GPU, at 0, 1, 3, 5, 8 and 12: 96
// requests 532 522 497 479 481 489 us; verify windows 106 86 71 69 74 79; the E4M3 batch 165 156 140 128 125 128).
template <bool kF8>
constexpr int kStartOf = kF8 ? 8 : 5;
constexpr float kUnset = -3.0e38f;           // a reference that no score has set
// Warps: the softmax groups, the one that finds the pieces and issues the scores' products, the one that
// issues the values', those that fetch.
template <int D, int N, bool kF8>
struct Roles {
  static constexpr int kCtas = N == 16 && (kF8 || D == 64) ? 2 : 1;  // blocks of an SM
  // At 16 rows two groups take tiles in turn, each with sums and references of its own, added at the end of
  // a piece; else a group takes 16 of the rows.
  static constexpr int kTurns = N == 16 && kCtas == 1 ? 2 : 1;
  static constexpr int kGroups = N / kCols * kTurns, kSoft = kGroups * kGroup;
  static constexpr int kFetch = 64;  // threads that fetch
  static constexpr int kScoreWarp = kSoft / 32, kValueWarp = kScoreWarp + 1, kFetchWarp = kValueWarp + 1;
  static constexpr int kT = 32 * kFetchWarp + kFetch;
  static constexpr int kReaders = kSoft / 32 + 1 + kFetch / 32;  // warps that read a piece
};
constexpr int kMostTokens = 0x7fffffff - 1024;  // of a request: a tile behind them is still an int
constexpr int kMaxBlocks = 304;              // blocks of a launch at most
// Powers of two that a weight may pass its reference by. E4M3: its f16 number is at most 2^(7 + 7), so that what two
// of its parts leave, below 2^8, times 2^8 is an f16 number (from 18688 on it was not: infinite, and the row NaN).
template <bool kF8>
constexpr float kHead = kF8 ? 7.0f : 8.0f;
// The largest value scale (E4M3). Where scales are 2^L the references are higher by L, and the sum, of probabilities
// alone, begins at 2^-L: what fp32 drops of it, below 2^-126, is then less than 2^-46 of the largest.
constexpr float kMostScale = 1.2089258196146292e24f;  // 2^80

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
  int32_t* count;   // [kMaxBlocks][N / 16], zero between calls
  float2* ml;       // [2 kMaxBlocks][rows of a unit]: reference (base 2) and sum
  float* acc;       // [2 kMaxBlocks][rows of a unit][D]
  int32_t* dev_status;
  tfd_kv_pages c;
  int rows, q_heads, group, max_pages, requests, max_new, window, qk;
  float eps, scale;  // scale: times log2 e
  uint32_t page_mul, page_shift;  // token / page_size = 2 token * page_mul >> (32 + page_shift)
  int page_stride, token_stride, head_stride;  // the cache's
  RopeTurns<D> turns;
};

// ---- PTX -----------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t sa(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
// The barrier gets this thread's arrival when all copies that it has issued are there.
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void bar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t par) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(par)
      : "memory");
  return ok;
}
__device__ __forceinline__ uint64_t now() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Bounded wait for the phase of parity `par` (about a second of global time); false on timeout.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t par) {
  if (bar_test(bar, par)) return true;
  uint64_t t0 = 0;
  for (int it = 1;; ++it) {
    if (bar_test(bar, par)) return true;
    if (it % 64 == 0) {
      const uint64_t t = now();
      if (t0 == 0) t0 = t;
      else if (t - t0 > 1000000000ull) return false;
    }
  }
}
// A barrier of some warps, the OR of a predicate over it, and an arrival that does not wait.
template <int kThreads>
__device__ __forceinline__ void warps_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}
template <int kThreads>
__device__ __forceinline__ void warps_arrive(int id) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}
template <int kThreads>
__device__ __forceinline__ bool warps_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "n"(kThreads)
      : "memory");
  return r;
}
// Shared-memory matrix descriptors: strides in bytes between a tile's pieces. 128-byte swizzle (2) or
// none (0).
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lead, uint32_t stride, int swizzle) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(stride >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)swizzle << 61;
}
// Instruction descriptor: fp32 accumulator, operands of types ta and tb (kind::f16: bf16 1; kind::f8f6f4:
// E4M3 0, E5M2 1), 128 x n; which are MN-major.
__device__ __forceinline__ uint32_t idesc(int n, uint32_t ta, uint32_t tb, bool mn_a, bool mn_b) {
  return (1u << 4) | (ta << 7) | (tb << 10) | ((uint32_t)mn_a << 15) | ((uint32_t)mn_b << 16) |
         ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
template <bool kF8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool acc) {
  if (kF8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"((uint32_t)acc)
        : "memory");
  else
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
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {  // not waited for
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// Waits for the loads; no use of the values moves before it.
template <int C>
__device__ __forceinline__ void tmem_ld_wait(float (&v)[C]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < C; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15};" ::"f"(v[0]),
      "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]),
      "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
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
// Two floats as E4M3 codes (nearest, saturating), and back.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3_floats(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<__half2*>(&r));
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t sub16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t mul16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// A product's high and low part. Where the high one is infinite the low one may be the other infinity, or zero
// times one: NaN, and the sum is the high part's.
__device__ __forceinline__ float add_low(float high, float low) {
  const float x = high + low;
  return x == x ? x : high;
}
// The largest of three; NaN if one is.
__device__ __forceinline__ float nan_or_most(float x, float y, float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
// The largest of a warp's values (NaN passed over), in all lanes.
__device__ __forceinline__ float warp_most(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ bool finite_(float x) { return fabsf(x) < INFINITY; }
// l 2^e, e <= 0, also where 2^e is below fp32's range and l is large.
__device__ __forceinline__ float lowered(float l, float e) {
  return l * exp2_(fmaxf(e, -100.0f)) * exp2_(fminf(e + 100.0f, 0.0f));
}

// A token's place in its request's table.
template <int D>
__device__ __forceinline__ int page_of(const Args<D>& a, int64_t token) {
  return (int)(__umulhi(2u * (uint32_t)token, a.page_mul) >> a.page_shift);
}

// a / b of numbers that rarely need 64 bits.
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  return ((uint64_t)a | (uint64_t)b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// ---- the line ------------------------------------------------------------------------------------
struct Request {
  int r, row0, n, len;   // its rows and the tokens before them
  int64_t base;          // first tile of its first unit on the line
  int tile0, tiles, mt;  // first tile of its tokens that a row can see, tiles from there, units a head
  int places;            // of a unit on the line
  bool bad;
};

// The first token that a row behind `len` tokens can see (with `tree` one that sees no new token is a depth back).
template <int D>
__device__ __forceinline__ int first_seen(const Args<D>& a, int len) {
  return a.window >= 0 ? (int)max((int64_t)0, (int64_t)len - a.window - (a.tree ? 1 : 0)) : 0;
}

// Request r's part of the line.
template <int D, int N, bool kF8>
__device__ __forceinline__ Request request(const Args<D>& a, int r) {
  Request q;
  q.r = r;
  q.row0 = a.row_start[r];
  const int64_t n = (int64_t)a.row_start[r + 1] - q.row0;
  q.len = a.lens[r];
  q.base = 0;
  q.bad = q.row0 < 0 || n < 0 || n > a.max_new || q.row0 + n > a.rows || q.len < 0 ||
          (n > 0 && (q.len + n > (int64_t)a.max_pages * a.c.page_size || q.len + n > kMostTokens));
  q.n = q.bad ? 0 : (int)n;
  q.tile0 = q.n > 0 ? first_seen(a, q.len) / kTile : 0;
  q.tiles = q.n > 0 ? (q.len + q.n - 1) / kTile + 1 - q.tile0 : 0;
  q.mt = (q.n * a.group + N - 1) / N;
  q.places = q.tiles + kStartOf<kF8>;
  return q;
}

// A unit's part in a block's stretch of the line: what everyone needs to know of it.
struct Piece {
  int64_t line0;          // the unit's first tile on the line
  int r, row0, n, len;    // request; its rows and the tokens before them
  int tile0, tiles;       // the unit's first tile of tokens, its tiles
  int first, cnt;         // of these the piece's: from, number (0: no more pieces)
  int h, valid;           // head; (row, query head) pairs there are
  int j0, h0;             // the first pair's row and query head within the group
};

// A block's odds and ends.
struct Misc {
  Request first;  // the request in which the block's cut falls
  int64_t ends[2];
  Piece piece[kAhead];
  int last[4], odd[4];
  uint32_t tmem;
};

// Cuts of the line, on which a unit of `tiles` takes kStart places and one for each tile. A cut falls every
// `share` places, but not within `keep` tiles of a unit's ends (there it moves to that end), nor in a unit of
// fewer than `least`.
template <int kStart>
struct Cuts {
  int64_t share;
  int keep, least;
  // the block that has the first tile of the unit that begins at `line0`
  __device__ __forceinline__ int64_t owner(int64_t line0, int tiles) const {
    return quot(line0 + kStart + (tiles < least ? tiles : keep) - 1, share);
  }
  __device__ __forceinline__ int64_t pieces(int64_t line0, int tiles) const {
    if (tiles < least) return 1;
    return quot(line0 + kStart + tiles - keep, share) - owner(line0, tiles) + 1;
  }
  // where the cut at `t`, which lies in the unit, moves to
  __device__ __forceinline__ int64_t moved(int64_t t, int64_t line0, int tiles) const {
    const int64_t at = t - line0 - kStart;
    if (tiles < least || at < keep) return line0;
    return at > tiles - keep ? line0 + kStart + tiles : t;
  }
};

// Parts that a value of q' or a weight enters its products in, side by side as columns: two bf16 ones
// against bf16 keys and values; four of 8 bits against E4M3 (q' in E4M3, weights in E5M2), of which the last two
// stand for 2^-8 of what they are.
template <int D, int N, bool kF8>
struct Smem {
  static constexpr int kParts = kF8 ? 4 : 2;
  static constexpr int kSlot = kF8 ? kTile * 128 : kTile * D * 2;  // E4M3: rows of 128 bytes, whatever D is
  static constexpr bool kTwo = Roles<D, N, kF8>::kCtas == 2;  // blocks an SM
  static constexpr int kSlots = kTwo ? 5 : kF8 ? 11 : D == 64 ? 9 : N == 64 ? 5 : 6;  // keys, values in turn
  static constexpr int kQ = kSlots * kSlot;                  // q': [row bytes / 128][parts N] rows of 128 bytes
  static constexpr int kQBytes = kF8 ? 512 * N : 4 * N * D;
  static constexpr int kQs = kTwo ? 2 : 1;                   // of them: the next piece's is made ahead
  static_assert(kQs == 1 || Roles<D, N, kF8>::kTurns == 1, "made after the piece's first tile, which the group has");
  static constexpr int kP = kQ + kQs * kQBytes;              // weights: [parts N / (16 bytes)][128] x 16 bytes
  static constexpr int kTurns = Roles<D, N, kF8>::kTurns, kPlace = 4 * N * kTile;  // a place for weights a turn
  static constexpr int kRows = kP + kTurns * kPlace;         // two of: what each row sees: from where, which new
  static constexpr int kRef = kRows + 2 * N * 8;             // reference of each row
  static constexpr int kFac = kRef + kTurns * N * 4;
  static constexpr int kFac2 = kFac + kTurns * N * 4;        // E4M3: what a factor is below 2^-100
  static constexpr int kRed = kFac2 + (kF8 ? N * 4 : 0);    // [groups][4][16]
  static constexpr int kPow = kRed + kTurns * N * 16;        // E4M3: two of: the power of two of q' of each row
  static constexpr int kBars = kPow + (kF8 ? 2 * N * 4 : 0);
  static constexpr int kMisc = (kBars + 8 * (2 * kSlots + 13 + 2 * kAhead) + 15) / 16 * 16;
  static constexpr int kBytes = kMisc + (int)sizeof(Misc);
  static_assert(kBytes <= (kTwo ? 113 : 227) * 1024, "shared memory of a block");
  static constexpr uint32_t kWide = kParts * N;              // columns of a product
  static constexpr uint32_t kO = 2 * kWide;                  // scores twice, then the weighted values a turn
  static constexpr uint32_t kUsed = kO + kTurns * kWide;
  static constexpr uint32_t kTmem = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static_assert(kUsed <= 512, "tensor memory");
};

// Sums of 16 columns over a warp: lanes 2 i and 2 i + 1 end with column i's in v[0].
__device__ __forceinline__ void column_sums(float (&v)[kCols]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 8, mask = 16; n > 0; n >>= 1, mask >>= 1) {
    const bool up = lane & mask;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
      }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
}

template <int D, int N, bool kF8>
__global__ void __launch_bounds__(Roles<D, N, kF8>::kT, Roles<D, N, kF8>::kCtas)
paged_attn_kernel(const __grid_constant__ Args<D> a) {
  using M = Smem<D, N, kF8>;
  using R = Roles<D, N, kF8>;
  constexpr int kFetch = R::kFetch, kT = R::kT, kScoreWarp = R::kScoreWarp;
  extern __shared__ __align__(1024) unsigned char sm[];  // all of the block's: it begins on a swizzle's period
  Misc& ms = *reinterpret_cast<Misc*>(sm + M::kMisc);
  int64_t* scan = reinterpret_cast<int64_t*>(sm + M::kP);  // before there are weights
  if (sa(sm) & 1023u) {
    if (threadIdx.x == 0) set_dev_status(a.dev_status, TFD_ERR_CUDA);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t bars = sa(sm + M::kBars);
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (M::kSlots + s); };
  const uint32_t more = bars + 16u * M::kSlots;
  auto s_full = [&](int b) { return more + 8u * b; };
  auto s_empty = [&](int b) { return more + 16u + 8u * b; };
  auto p_full = [&](int t) { return more + 32u + 8u * t; };
  auto p_empty = [&](int t) { return more + 48u + 8u * t; };
  const uint32_t q_full = more + 64u, o_full = more + 72u, o_empty = more + 80u, drained = more + 88u;
  auto w_full = [&](int e) { return more + 104u + 8u * e; };
  auto w_empty = [&](int e) { return more + 104u + 8u * (kAhead + e); };
  constexpr int kTurns = R::kTurns;
  auto round_of = [](int64_t g) { return (uint32_t)(g / kTurns); };  // tile g's, of its turn g mod kTurns
  if (tid == 0) {
    for (int s = 0; s < M::kSlots; ++s) {
      bar_init(full(s), kFetch);
      bar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(s_full(b), 1);
      bar_init(s_empty(b), R::kSoft / kTurns);
      bar_init(p_full(b), R::kSoft / kTurns);
      bar_init(p_empty(b), 1);
    }
    bar_init(q_full, R::kSoft / kTurns);
    bar_init(o_full, 1);
    bar_init(o_empty, R::kSoft);
    bar_init(drained, 1);
    bar_init(drained + 8u, 1);
    for (int e = 0; e < kAhead; ++e) {
      bar_init(w_full(e), 1);
      bar_init(w_empty(e), R::kReaders);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int i = 0; i < 4; ++i) ms.odd[i] = 0;
  }
  constexpr uint32_t kTmem = M::kTmem, kO = M::kO, kWide = M::kWide;
  if (warp == kScoreWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&ms.tmem)),
                 "r"(kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tfd_host::after_previous();
  const int H = a.c.heads, ps = a.c.page_size;

  // ---- this block's stretch of the line -----------------------------------------------------------
  int64_t total = 0;
  constexpr int kStart = kStartOf<kF8>;
  Cuts<kStart> cuts;
  {
    const int per = (a.requests + kT - 1) / kT;
    const int r0 = min(a.requests, tid * per), r1 = min(a.requests, r0 + per);
    int64_t mine = 0;
    Request q0 = {};  // this thread's first
    if (tid < 2) ms.ends[tid] = -1;
    for (int r = r0; r < r1; ++r) {
      const Request q = request<D, N, kF8>(a, r);
      if (r == r0) q0 = q;
      if (q.bad && blockIdx.x == 0) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
      mine += (int64_t)q.places * q.mt * H;
    }
    int64_t x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t lo = __shfl_up_sync(0xffffffffu, (uint32_t)x, d);
      const uint32_t hi = __shfl_up_sync(0xffffffffu, (uint32_t)((uint64_t)x >> 32), d);
      if (lane >= d) x += (int64_t)((uint64_t)hi << 32 | lo);
    }
    if (lane == 31) scan[warp] = x;
    fence_before();
    __syncthreads();
    fence_after();
    int64_t before = x - mine;
    for (int w = 0; w < kT / 32; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    cuts.share = quot(total + gridDim.x - 1, gridDim.x);
    cuts.keep = (int)min(cuts.share, (int64_t)kKeep);
    cuts.least = (int)min(2 * cuts.share, (int64_t)kLeast);
    // the block's stretch: from its cut to the next one's
    int64_t at = before;
    for (int r = r0; r < r1; ++r) {  // for the threads in whose requests a cut falls
      const int64_t lo = blockIdx.x * cuts.share, hi = lo + cuts.share;
      if (!((before <= lo && lo < before + mine) || (before <= hi && hi < before + mine))) break;
      Request q = r == r0 ? q0 : request<D, N, kF8>(a, r);
      const int64_t u = (int64_t)q.places * q.mt * H;
      q.base = at;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t t = e ? hi : lo;
        if (at <= t && t < at + u) {
          ms.ends[e] = cuts.moved(t, at + quot(t - at, q.places) * q.places, q.tiles);
          if (e == 0) ms.first = q;
        }
      }
      at += u;
    }
    __syncthreads();
  }
  const uint32_t tmem = ms.tmem;
  const int64_t t0 = ms.ends[0] < 0 ? total : ms.ends[0], t_end = ms.ends[1] < 0 ? total : ms.ends[1];
  const int64_t steps = t_end - t0;  // places of the stretch, some of them tiles
  bool ok = true;                   // none of this thread's waits has run out

  // Piece k of the stretch, from the warp that finds them: a copy. All lanes of a warp call it.
  auto get_piece = [&](int k, bool one_lane) {
    const int e = k % kAhead;
    if (ok) ok = bar_wait(w_full(e), (uint32_t)(k / kAhead) & 1u);
    if (!one_lane) ok = __all_sync(0xffffffffu, ok);
    Piece p = ms.piece[e];
    if (!ok) p.cnt = 0;
    if (!one_lane) __syncwarp();
    if (one_lane || lane == 0) bar_arrive(w_empty(e));
    return p;
  };

  if (steps > 0 && warp >= R::kFetchWarp) {
    // ---- fetch: a warp half of each tile, a lane the pages of two tokens ----------------------------
    constexpr int kMine = kTile / (kFetch / 32), kPer = kMine / 32;  // tokens of a warp, of a lane
    constexpr int es = kF8 ? 1 : 2, L = D * es / 16, P = 32 / L;  // lanes of a vector, vectors a step
    const int mine0 = kMine * (warp - R::kFetchWarp), c = lane % L;
    const unsigned char* kbase = (const unsigned char*)a.c.k + 16 * c;
    const unsigned char* vbase = (const unsigned char*)a.c.v + 16 * c;
    // where this lane's pieces go: rows mine0 + lane / L + j P, whose swizzle repeats after 8 rows
    uint32_t to[8 / P];
#pragma unroll
    for (int u = 0; u < 8 / P; ++u) {
      const int row = mine0 + u * P + lane / L;
      to[u] = (uint32_t)((c >> 3) * (kTile * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
    }
    int slot = 0;
    uint32_t round = 0;  // of the slots
    for (int k = 0;; ++k) {
      const Piece w = get_piece(k, false);
      if (w.cnt == 0) break;
      const int tokens = w.len + w.n, low = first_seen(a, w.len);
      const int32_t* table = a.table + w.r * a.ldt;
      const int64_t head = (int64_t)w.h * a.head_stride;
      int64_t tok = (int64_t)(w.tile0 + w.first) * kTile + mine0 + lane;
      int pg[kPer], page[kPer];
      auto look_up = [&](bool on) {
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          pg[q] = page_of(a, tok + 32 * q);
          page[q] = on && tok + 32 * q >= low && tok + 32 * q < tokens ? table[pg[q]] : -1;
        }
      };
      look_up(true);
#pragma unroll 1
      for (int i = 0; i < w.cnt && ok; ++i) {
        int64_t off[kPer];
        uint32_t there[kPer];
        bool whole = true;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          const bool in = page[q] >= 0 && page[q] < a.c.pages;
          if (tok + 32 * q >= low && tok + 32 * q < tokens && !in)
            set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
          const int64_t at = (int64_t)((int)tok + 32 * q - pg[q] * ps) * a.token_stride;
          off[q] = in ? ((int64_t)page[q] * a.page_stride + at + head) * es : 0;
          there[q] = __ballot_sync(0xffffffffu, in);
          whole = whole && there[q] == 0xffffffffu;
        }
        tok += kTile;
        look_up(i + 1 < w.cnt);
        int64_t from[kMine / P];  // of the rows whose pieces this lane copies
#pragma unroll
        for (int j = 0; j < kMine / P; ++j)
          from[j] = __shfl_sync(0xffffffffu, off[j * P / 32], (j * P & 31) + lane / L);
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
          if (round > 0)
            ok = __all_sync(0xffffffffu, bar_wait(empty(slot), (round - 1) & 1u));
          if (!ok) break;
          const uint32_t st = sa(sm) + (uint32_t)slot * M::kSlot;
          const unsigned char* base = v ? vbase : kbase;
          if (whole) {
#pragma unroll
            for (int j = 0; j < kMine / P; ++j)
              copy16(st + to[j % (8 / P)] + j / (8 / P) * 1024, base + from[j], true);
          } else {
#pragma unroll
            for (int j = 0; j < kMine / P; ++j)
              copy16(st + to[j % (8 / P)] + j / (8 / P) * 1024, base + from[j],
                     (there[j * P / 32] >> ((j * P & 31) + lane / L)) & 1u);
          }
          copy_arrive(full(slot));
          if (++slot == M::kSlots) slot = 0, ++round;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (steps > 0 && tid == 32 * kScoreWarp) {
    // ---- the pieces, two ahead, and the scores' products: one thread --------------------------------
    Request rq = ms.first;
    int64_t t = t0;
    int found = 0;
    bool more_pieces = true;
    auto find = [&]() {
      Piece p;
      p.cnt = 0;
      while (t < t_end && t >= rq.base + (int64_t)rq.places * rq.mt * H) {
        const int64_t next = rq.base + (int64_t)rq.places * rq.mt * H;
        if (rq.r + 1 >= a.requests) t = t_end;  // lengths that changed meanwhile
        else rq = request<D, N, kF8>(a, rq.r + 1);
        rq.base = next;
      }
      if (t < t_end) {
        const int64_t unit = quot(t - rq.base, rq.places);
        p.line0 = rq.base + unit * rq.places;
        p.r = rq.r, p.row0 = rq.row0, p.n = rq.n, p.len = rq.len, p.tile0 = rq.tile0, p.tiles = rq.tiles;
        const int64_t line1 = p.line0 + kStart;  // of its first tile
        p.first = (int)max((int64_t)0, t - line1);
        p.h = (int)quot(unit, rq.mt);
        const int m0 = (int)(unit - (int64_t)p.h * rq.mt) * N;
        p.cnt = (int)(min((int64_t)rq.tiles, t_end - line1) - p.first);
        p.valid = min(N, rq.n * a.group - m0);
        p.j0 = m0 / a.group;
        p.h0 = m0 - p.j0 * a.group;
        t = line1 + p.first + p.cnt;
      }
      const int e = found % kAhead;
      if (found >= kAhead && ok) ok = bar_wait(w_empty(e), (uint32_t)(found / kAhead - 1) & 1u);
      if (!ok) return;
      ms.piece[e] = p;
      bar_arrive(w_full(e));
      ++found;
      more_pieces = p.cnt > 0;
    };
    const uint32_t desc = idesc(kWide, kF8 ? 0 : 1, kF8 ? 0 : 1, false, false);
    constexpr int kStep = kF8 ? 32 : 16;  // k of a product: 32 bytes of a row of dims
    const uint64_t keys = sdesc(sa(sm), 16, 1024, 2), rows = sdesc(sa(sm + M::kQ), 16, 1024, 2);
    for (int i = 0; i < kAhead && ok && more_pieces; ++i) find();
    uint32_t slot = 0, round = 0, g = 0;
    for (int p = 0; ok; ++p) {
      const int cnt = ms.piece[p % kAhead].cnt;
      if (cnt == 0) break;
      ok = bar_wait(q_full, (uint32_t)p & 1u);
      const uint64_t q0 = rows + (uint32_t)(p % M::kQs * (M::kQBytes / 16));
      for (int i = 0; i < cnt && ok; ++i, ++g) {
        const uint32_t b = g & 1;
        if (g >= 2) ok = bar_wait(s_empty(b), ((g >> 1) - 1) & 1u);
        if (ok) ok = bar_wait(full(slot), round & 1u);
        if (!ok) break;
        fence_async();
        fence_after();
        const uint64_t k0 = keys + slot * (M::kSlot / 16);
#pragma unroll
        for (int k = 0; k < D / kStep; ++k)
          mma<kF8>(tmem + b * kWide, k0 + (uint32_t)((k >> 2) * (kTile * 8) + (k & 3) * 2),
                   q0 + (uint32_t)((k >> 2) * (kWide * 8) + (k & 3) * 2), desc, k != 0);
        if (!TFD_TEST_STALL_EXCHANGE) mma_commit(s_full(b));
        mma_commit(empty(slot));
        slot += 2;
        if (slot >= M::kSlots) slot -= M::kSlots, ++round;
        if (i == min(cnt, 2) - 1)
          while (ok && more_pieces && found < p + 1 + kAhead) find();
      }
    }
    mma_commit(drained);  // no product may still read or write when this block's memory is given back
    if (!bar_wait(drained, 0)) ok = false;
  } else if (steps > 0 && tid == 32 * R::kValueWarp) {
    // ---- the values' products: one thread ------------------------------------------------------------
    const uint32_t desc = idesc(kWide, kF8 ? 0 : 1, 1, true, true);
    constexpr int kStep = kF8 ? 32 : 16;  // tokens of a product
    // values: 64 dims (E4M3: 128) a row of 128 bytes; heads of 64 leave the other 64 rows to themselves
    const uint64_t values = sdesc(sa(sm), D == 64 || kF8 ? 0 : kTile * 128, 1024, 2);
    const uint64_t weights = sdesc(sa(sm + M::kP), 128, kTile * 16, 0);
    uint32_t slot = 1, round = 0, g = 0;
    for (int p = 0;; ++p) {
      const Piece w = get_piece(p, true);
      if (w.cnt == 0) break;
      if (p > 0) ok = bar_wait(o_empty, (uint32_t)(p - 1) & 1u);
      for (int i = 0; i < w.cnt && ok; ++i, ++g) {
        const uint32_t turn = g % kTurns;
        ok = bar_wait(p_full(turn), (g / kTurns) & 1u) && bar_wait(full(slot), round & 1u);
        if (!ok) break;
        fence_async();
        fence_after();
        const uint64_t v0 = values + slot * (M::kSlot / 16), p0 = weights + turn * (M::kPlace / 16);
#pragma unroll
        for (int k = 0; k < kTile / kStep; ++k)
          mma<kF8>(tmem + kO + turn * kWide, v0 + (uint32_t)(k * kStep * 8), p0 + (uint32_t)(k * kStep), desc,
                   i >= kTurns || k != 0);
        mma_commit(empty(slot));
        mma_commit(p_empty(turn));
        if (i == w.cnt - 1) mma_commit(o_full);
        slot += 2;
        if (slot >= M::kSlots) slot -= M::kSlots, ++round;
      }
      if (!ok) break;
    }
    mma_commit(drained + 8u);
    if (!bar_wait(drained + 8u, 0)) ok = false;
  } else if (steps > 0 && warp < kScoreWarp) {
    // ---- softmax of 16 rows: a thread a token; then their sums, a thread a dim -----------------------
    const int grp = warp / 4, bid = 1 + grp, gw = warp & 3, gt = tid & (kGroup - 1);
    const int turn = kTurns == 1 ? 0 : grp, n0 = kTurns == 1 ? grp * kCols : 0;
    constexpr int kBoth = kTurns * kGroup, kBothId = 8, kSumId = 9;  // barriers of groups that share rows
    float* s_ref = reinterpret_cast<float*>(sm + M::kRef) + grp * kCols;
    float* s_fac = reinterpret_cast<float*>(sm + M::kFac) + grp * kCols;
    float* s_fac2 = reinterpret_cast<float*>(sm + M::kFac2) + grp * kCols;
    float* s_red = reinterpret_cast<float*>(sm + M::kRed) + 4 * grp * kCols;
    unsigned char* s_p = sm + M::kP + turn * M::kPlace;
    const uint32_t o_at = kO + turn * kWide, lanes = (uint32_t)(32 * gw) << 16;
    // what the unit's rows of piece p see: the first cached token, the new ones
    auto rows_of = [&](int p) { return reinterpret_cast<int2*>(sm + M::kRows) + (p & 1) * N; };
    auto sees = [&](const int2& row, int key, int len) {
      const int j = key - len;
      return j < 0 ? key >= row.x : j < 32 && (((uint32_t)row.y >> (j & 31)) & 1u);
    };
    // from where all the unit's rows see the cached tokens, and the new ones that they all see
    int2 every = make_int2(0, 0), every_next = every;

    // q' of a piece in two parts, and what each of its rows sees; the rows' q is loaded before. Four rows
    // a warp at once, 8 lanes a row: a lane holds the first and second elements of D / 16 pairs.
    constexpr int E = D / 16;
    uint32_t raw[E], gam[E], raw_word = 0u;
    int raw_pos = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
      gam[e] = a.gamma && (a.qk & TFD_QK_NORM)
                   ? (uint32_t)a.gamma[(2 * e / E) * (D / 2) + E * (lane & 7) + 2 * e % E] |
                         (uint32_t)a.gamma[(2 * e / E) * (D / 2) + E * (lane & 7) + 2 * e % E + 1] << 16
                   : 0x3F803F80u;
    auto load_q = [&](const Piece& w) {
      if (lane < w.n) {
        if (a.tree) raw_word = (uint32_t)a.tree[w.row0 + lane];
        if (a.pos && (a.qk & TFD_QK_ROPE)) raw_pos = a.pos[w.row0 + lane];
      }
      if (turn > 0) return;  // the first group makes q' for both
      const int v = w.h0 + min(n0 + 4 * gw + lane / 8, w.valid - 1), j = v / a.group;
      const uint16_t* src = a.q + (w.row0 + w.j0 + j) * a.ldq + (int64_t)(w.h * a.group + v - j * a.group) * D +
                            E * (lane & 7);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (E == 8) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + half * (D / 2));
          raw[half * (E / 2)] = x.x, raw[half * (E / 2) + 1] = x.y;
          raw[half * (E / 2) + E / 2 - 2] = x.z, raw[half * (E / 2) + E / 2 - 1] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(src + half * (D / 2));
          raw[half * (E / 2)] = x.x, raw[half * (E / 2) + 1] = x.y;
        }
      }
    };
    auto prepare = [&](const Piece& w, int p) {
      int2* s_rows = rows_of(p) + n0;
      // new row `lane`: its word, depth and position
      const bool there = lane < w.n;
      const uint32_t rows_there = w.n == 32 ? 0xffffffffu : (1u << w.n) - 1u;
      uint32_t words = (2u << lane) - 1u;  // itself and those before
      if (a.tree && there) words = raw_word;
      words &= rows_there;
      const int depths = w.len + (a.tree ? __popc(words) - 1 : lane);
      int places = there && a.pos && (a.qk & TFD_QK_ROPE) ? raw_pos : depths;
      if (places < 0) {
        if (there && a.pos && (a.qk & TFD_QK_ROPE)) set_dev_status(a.dev_status, TFD_ERR_DEVICE_DATA);
        places = 0;
      }
      {
        const bool in = lane >= w.j0 && lane <= w.j0 + (w.h0 + w.valid - 1) / a.group;  // the unit's
        const int deepest = __reduce_max_sync(0xffffffffu, in ? depths : INT32_MIN);
        const int64_t from = a.window >= 0 ? (int64_t)deepest - a.window : -1;
        every_next.x = from > 0 ? (int)min(from, (int64_t)w.len) : 0;
        every_next.y = (int)(__reduce_and_sync(0xffffffffu, in ? words : 0xffffffffu) &
                             __ballot_sync(0xffffffffu, depths >= from));
      }
      if (turn > 0) return;
      const int i = 4 * gw + lane / 8, n = n0 + i, l = lane & 7;
      const bool row = n < w.valid;
      const int j = w.j0 + (w.h0 + min(n, w.valid - 1)) / a.group;
      float x[2 * E];  // first elements of the pairs, then the second
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[2 * e] = row ? bf16_lo(raw[e]) : 0.0f;
        x[2 * e + 1] = row ? bf16_hi(raw[e]) : 0.0f;
      }
      if (a.qk & TFD_QK_NORM) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int m = 4; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float inv = row ? 1.0f / sqrtf(ss / (float)D + a.eps) : 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          x[2 * e] = x[2 * e] * inv * bf16_lo(gam[e]);
          x[2 * e + 1] = x[2 * e + 1] * inv * bf16_hi(gam[e]);
        }
      }
      if (a.qk & TFD_QK_ROPE) {
        const int at = __shfl_sync(0xffffffffu, places, j);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float sn, cs;
          rope_pair_fast<D>(at, a.turns, E * l + e, sn, cs);
          const float first = x[e], second = x[E + e];
          x[e] = first * cs - second * sn;
          x[E + e] = first * sn + second * cs;
        }
      }
      // the new tokens that the row sees, and its first cached one
      const uint32_t word = __shfl_sync(0xffffffffu, words, j);
      const int64_t from = a.window >= 0 ? (int64_t)__shfl_sync(0xffffffffu, depths, j) - a.window : -1;
      uint32_t sees = word;
      if (a.window >= 0) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t deep = __ballot_sync(0xffffffffu, depths >= __shfl_sync(0xffffffffu, from, 8 * r));
          if (lane / 8 == r) sees &= deep;
        }
      }
      // past the last row: it hides nothing
      if (l == 0)
        s_rows[i] = row ? make_int2(from > 0 ? (int)min(from, (int64_t)w.len) : 0, (int)sees) : make_int2(0, -1);
      if (kF8) {
        // into E4M3's range, the row's largest magnitude in [128, 256); then part by part what is left
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) {
          x[e] *= a.scale;
          top = fmaxf(top, fabsf(x[e]));
        }
#pragma unroll
        for (int m = 4; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        int ex = (int)((__float_as_uint(top) >> 23) & 0xffu) - 127 - 7;
        ex = finite_(top) ? max(-126, min(120, ex)) : 0;
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
        if (l == 0)
          reinterpret_cast<float*>(sm + M::kPow)[(p & 1) * N + n] =  // infinite: NaN, as the formula gives
              finite_(top) ? __uint_as_float((uint32_t)(127 + ex) << 23) : NAN;
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) x[e] *= down;
#pragma unroll
        for (int part = 0; part < 4; ++part)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w[E / 4];
#pragma unroll
            for (int e = 0; e < E; e += 4) {
              float* y = x + half * E + e;
              const uint32_t lo = e4m3x2(y[0], y[1]), hi = e4m3x2(y[2], y[3]);
              w[e / 4] = lo | hi << 16;
              const float2 b0 = e4m3_floats(lo), b1 = e4m3_floats(hi);
              const float up = part == 1 ? 256.0f : 1.0f;
              y[0] = (y[0] - b0.x) * up, y[1] = (y[1] - b0.y) * up;
              y[2] = (y[2] - b1.x) * up, y[3] = (y[3] - b1.y) * up;
            }
            const int d = half * (D / 2) + E * l, r = part * N + n;
            unsigned char* to =
                sm + M::kQ + p % M::kQs * M::kQBytes + r * 128 + (((d >> 4) ^ (r & 7)) << 4) + (d & 15);
            if (E == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[E / 4 - 1]);
            else *reinterpret_cast<uint32_t*>(to) = w[0];
          }
      } else {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float y0 = x[half * E + e] * a.scale, y1 = x[half * E + e + 1] * a.scale;
            hi[e / 2] = bf16x2(y0, y1);
            const float b0 = bf16_lo(hi[e / 2]), b1 = bf16_hi(hi[e / 2]);
            lo[e / 2] = bf16x2(finite_(b0) ? y0 - b0 : 0.0f, finite_(b1) ? y1 - b1 : 0.0f);
          }
          const int d = half * (D / 2) + E * l;
          unsigned char* to = sm + M::kQ + p % M::kQs * M::kQBytes + (d >> 6) * (kWide * 128) + n * 128 +
                              ((((d >> 3) & 7) ^ (n & 7)) << 4) + (d & 7) * 2;
          if (E == 8) {
            *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[E / 2 - 2], hi[E / 2 - 1]);
            *reinterpret_cast<uint4*>(to + N * 128) = make_uint4(lo[0], lo[1], lo[E / 2 - 2], lo[E / 2 - 1]);
          } else {
            *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(to + N * 128) = make_uint2(lo[0], lo[1]);
          }
        }
      }
      fence_async();
      bar_arrive(q_full);
    };

    int64_t g0 = 0;  // tiles before the piece's
    Piece next = get_piece(0, false);
    // decided by all that share rows: they wait for each other
    auto any = [&](bool x) {
      return kTurns == 1 ? warps_any<kGroup>(bid, x) : warps_any<kBoth>(kBothId, x);
    };
    bool have = !any(next.cnt == 0);
    if (have) {
      load_q(next);
      prepare(next, 0);
    }
    for (int p = 0; have; ++p) {
      const Piece cur = next;
      const int tokens = cur.len + cur.n;
      warps_sync<kGroup>(bid);  // the last piece's sums are done with
      if (gt < kCols) s_ref[gt] = kUnset;
      warps_sync<kGroup>(bid);  // what each row sees, and its reference
      const int2* s_rows = rows_of(p) + n0;
      if (tid == 0) ms.odd[(p + 2) & 3] = 0;
      if (kTurns > 1 && turn > 0 && p > 0) warps_sync<kBoth>(kSumId);  // its last sums have been fetched
      every = every_next;
      float sum[kCols];
#pragma unroll
      for (int n = 0; n < kCols; ++n) sum[n] = 0.0f;
      const int32_t* table = a.table + cur.r * a.ldt;
      const int i0 = kTurns == 1 ? 0 : (int)((turn + g0) & 1);  // this group's first tile of the piece
      int64_t tok = (int64_t)(cur.tile0 + cur.first + i0) * kTile + gt;
      // of this thread's token; -1: none. In a unit's first tile also of tokens left of every row's window, whose
      // entries may name any page: what is read of it is masked (to leave them out here took 4% of an E4M3 batch)
      auto page_at = [&](int64_t tok, int i) {
        return i < cur.cnt && tok < tokens ? table[page_of(a, tok)] : -1;
      };
      int page = page_at(tok, i0), page_next = page_at(tok + kTurns * kTile, i0 + kTurns);
      float ks = 0.0f, vs = 1.0f, ks_next = 0.0f, vs_next = 1.0f;  // E4M3: its scales
      auto load_scales = [&](int64_t tok, int page, float& ks, float& vs) {
        ks = 0.0f, vs = 1.0f;
        if (page >= 0 && page < a.c.pages) {
          const int64_t at = (int64_t)page * (H * ps) + (cur.h * ps + (int)tok - page_of(a, tok) * ps);
          ks = a.c.k_scales[at];
          vs = a.c.v_scales[at];
        }
      };
      if (kF8) load_scales(tok, page, ks_next, vs_next);
      next = get_piece(p + 1, false);
      if (next.cnt > 0) load_q(next);

#pragma unroll 1
      for (int i = i0; i < cur.cnt; i += kTurns) {
        const int64_t g = g0 + i;
        const int b = (int)(g & 1);
        const int key0 = (cur.tile0 + cur.first + i) * kTile, key = key0 + gt;
        const bool there = page >= 0 && page < a.c.pages;
        tok += kTurns * kTile;
        page = page_next;
        page_next = page_at(tok + kTurns * kTile, i + 2 * kTurns);
        if (kF8) {
          ks = ks_next, vs = vs_next;
          load_scales(tok, page, ks_next, vs_next);
        }
        if (ok) ok = bar_wait(s_full(b), (uint32_t)(g >> 1) & 1u);
        fence_after();
        const bool partly = key0 < every.x || key0 + kTile > cur.len;  // the same for all groups
        float s[kCols];
        {
          float rest[kCols], more[kF8 ? 2 * kCols : 1];
          tmem_ld16(tmem + lanes + b * kWide + n0, s);
          tmem_ld16(tmem + lanes + b * kWide + N + n0, rest);
          if (kF8) {
            tmem_ld16(tmem + lanes + b * kWide + 2 * N + n0, more);
            tmem_ld16(tmem + lanes + b * kWide + 3 * N + n0, more + (kF8 ? kCols : 0));
          }
          tmem_ld_wait(s);
          tmem_ld_wait(rest);
          if (kF8) tmem_ld_wait(more);
          fence_before();
          bar_arrive(s_empty(b));
          if (kF8) {
#pragma unroll
            for (int n = 0; n < kCols; ++n)
              s[n] = fmaf(more[kF8 ? n : 0] + more[kF8 ? kCols + n : 0], 0.00390625f, s[n] + rest[n]);
          } else {
            // as add_low, looking at all sums before any (48 requests of 32 rows 1008 us, each by itself 1021, not at
            // all 1005; verify windows 69.1, 69.4 and 68.7)
            float odd = 0.0f;
#pragma unroll
            for (int n = 0; n < kCols; n += 2) odd = nan_or_most(odd, rest[n] += s[n], rest[n + 1] += s[n + 1]);
            if (odd != odd) {
#pragma unroll
              for (int n = 0; n < kCols; ++n) rest[n] = rest[n] == rest[n] ? rest[n] : s[n];
            }
#pragma unroll
            for (int n = 0; n < kCols; ++n) s[n] = rest[n];
          }
        }
        // E4M3: the value's scale is part of its weight, as the score's summand: the weights are at most 2^14. A sum
        // without them is at most 2^(96 + 7) a token; what a scale is below 2^-96 its weight is multiplied by
        float lv = 0.0f, lv_fin = 0.0f, small = 1.0f;
        if (kF8) {
          lv = fabsf(vs) <= kMostScale ? log2f(fabsf(vs)) : NAN;  // beyond: NaN for the rows that see it
          small = copysignf(1.0f, vs);
          if (fabsf(vs) < 1.262177448353619e-29f) {
            small = vs * 7.922816251426434e28f;
            lv = -96.0f;
          }
          lv_fin = finite_(lv) ? lv : 0.0f;
          const float* pow = reinterpret_cast<const float*>(sm + M::kPow) + (p & 1) * N + n0;
#pragma unroll
          for (int n = 0; n < kCols; n += 4) {
            const float4 f = *reinterpret_cast<const float4*>(pow + n);
            s[n] = fmaf(s[n] * f.x, ks, lv), s[n + 1] = fmaf(s[n + 1] * f.y, ks, lv);
            s[n + 2] = fmaf(s[n + 2] * f.z, ks, lv), s[n + 3] = fmaf(s[n + 3] * f.w, ks, lv);
          }
        }
        if (partly || !__all_sync(0xffffffffu, there)) {  // -inf where this token is not seen
#pragma unroll
          for (int n = 0; n < kCols; ++n)
            if (!there || !sees(s_rows[n], key, cur.len)) s[n] = -INFINITY;
        }
        bool free = g < kTurns;  // the weights' place
        auto wait_free = [&]() {
          if (!free && ok) ok = bar_wait(p_empty(turn), (round_of(g) - 1) & 1u);
          free = true;
        };
        float over = -INFINITY;  // by how much a score passes its reference
#pragma unroll
        for (int n = 0; n < kCols; n += 4) {
          const float4 r = *reinterpret_cast<const float4*>(s_ref + n);
          over = fmaxf(over, fmaxf(fmaxf(s[n] - r.x, s[n + 1] - r.y), fmaxf(s[n + 2] - r.z, s[n + 3] - r.w)));
        }
        if (i == i0 || warps_any<kGroup>(bid, over > kHead<kF8>)) {  // every row's reference is its largest score so far
          float most = 0.0f;
#pragma unroll
          for (int n = 0; n < kCols; ++n) {
            const float x = warp_most(s[n]);
            if (lane == n) most = x;
          }
          if (lane < kCols) s_red[gw * kCols + lane] = most;
          warps_sync<kGroup>(bid);
          if (gt < kCols) {
            const float was = s_ref[gt];
            const float x = fmaxf(fmaxf(fmaxf(s_red[gt], s_red[16 + gt]), fmaxf(s_red[32 + gt], s_red[48 + gt])),
                                  was);
            // E4M3, as two factors: a reference can rise with the values' scales where a sum is large (lowered; all
            // of that in each thread 131.9 us in a large batch, two factors 129.7, one 127.3)
            s_fac[gt] = exp2_(kF8 ? fmaxf(was - x, -100.0f) : was - x);
            if (kF8) s_fac2[gt] = exp2_(fminf(was - x + 100.0f, 0.0f));
            s_ref[gt] = x;
          }
          warps_sync<kGroup>(bid);
          if (i > i0) {
            wait_free();  // all so far is added up
            fence_after();
#pragma unroll 1
            for (int part = 0; part < M::kParts; ++part) {
              float o[kCols];
              tmem_ld16(tmem + lanes + o_at + part * N + n0, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int n = 0; n < kCols; ++n) o[n] *= kF8 ? s_fac[n] * s_fac2[n] : s_fac[n];
              tmem_st16(tmem + lanes + o_at + part * N + n0, o);
            }
            fence_before();
#pragma unroll
            for (int n = 0; n < kCols; ++n) sum[n] = kF8 ? sum[n] * s_fac[n] * s_fac2[n] : sum[n] * s_fac[n];
          }
        }
#pragma unroll
        for (int n = 0; n < kCols; n += 4) {
          const float4 r = *reinterpret_cast<const float4*>(s_ref + n);
          s[n] -= r.x, s[n + 1] -= r.y, s[n + 2] -= r.z, s[n + 3] -= r.w;
        }
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          if (kF8) {
            sum[n] += exp2_(s[n] - lv_fin);
            s[n] = exp2_(s[n] + 7.0f) * small;
          } else {
            s[n] = exp2_(s[n]);
            sum[n] += s[n];
          }
        }
        wait_free();
        if (kF8) {
          // f16 weights (2^-11) by bits: an E5M2 number is the upper half of an f16 one, and 3 of its 11
          // bits; what is left is exact, and four parts hold it all (of a number below 2^-12 all but 3 2^-24)
          uint32_t w[kCols / 2];
#pragma unroll
          for (int n = 0; n < kCols; n += 2) w[n / 2] = f16x2(s[n], s[n + 1]);
#pragma unroll
          for (int part = 0; part < 4; ++part) {
            uint32_t c[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) c[n] = __byte_perm(w[2 * n], w[2 * n + 1], 0x7531);
            *reinterpret_cast<uint4*>(s_p + ((part * N + n0) >> 4) * (kTile * 16) + gt * 16) =
                make_uint4(c[0], c[1], c[2], c[3]);
            if (part < 3) {
#pragma unroll
              for (int n = 0; n < kCols / 2; ++n) {
                w[n] = sub16x2(w[n], w[n] & 0xFF00FF00u);
                if (part == 1) w[n] = mul16x2(w[n], 0x5C005C00u);  // 256
              }
            }
          }
        } else {
#pragma unroll
          for (int n = 0; n < kCols; n += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = s[n + 2 * e], y = s[n + 2 * e + 1];
              hi[e] = bf16x2(x, y);
              lo[e] = bf16x2(x - bf16_lo(hi[e]), y - bf16_hi(hi[e]));
            }
            unsigned char* to = s_p + ((n0 + n) >> 3) * (kTile * 16) + gt * 16;
            *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(to + 2 * N * kTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        if (!kF8 && partly) {
          // a value that is not finite, of a token that not all rows see: 0 times it would be NaN. It
          // leaves the product, and is added at the end to the rows that see it. (E4M3 codes are not NaN;
          // to look for them here took 7% of a large batch's time.)
          const int64_t x = 2 * g + 1;
          const int slot = (int)(x % M::kSlots);
          if (there && !sees(every, key, cur.len)) {
            if (ok) ok = bar_wait(full(slot), (uint32_t)(x / M::kSlots) & 1u);
            auto at = [&](int c) {
              return reinterpret_cast<uint4*>(sm + slot * M::kSlot + (c >> 3) * (kTile * 128) + gt * 128 +
                                              (((c & 7) ^ (gt & 7)) << 4));
            };
            bool odd = false;
#pragma unroll 8
            for (int c = 0; c < D / 8; ++c) {
              const uint4 v = *at(c);
              const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                odd |= (u[e] & 0x7F80u) == 0x7F80u || (u[e] & 0x7F800000u) == 0x7F800000u;
            }
#pragma unroll 1
            for (int c = 0; odd && c < D / 8; ++c) {
              uint4 v = *at(c);
              uint32_t* u = &v.x;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((u[e] & 0x7F80u) == 0x7F80u) u[e] &= 0xFFFF0000u;
                if ((u[e] & 0x7F800000u) == 0x7F800000u) u[e] &= 0xFFFFu;
              }
              *at(c) = v;
            }
            // such tiles are among the unit's first two and last two
            const int at_tile = cur.first + i;
            const int bit = at_tile < 2 && key0 < every.x ? at_tile : 2 + cur.tiles - 1 - at_tile;
            if (odd) atomicOr(&ms.odd[p & 3], 1 << bit);
          }
        }
        fence_async();
        bar_arrive(p_full(turn));
        if (M::kQs > 1 && i == i0 && next.cnt > 0) prepare(next, p + 1);
      }
      g0 += cur.cnt;

      // ---- the sums; the next piece's scores can begin meanwhile ---------------------------------------
      const float mine_ref = gt < kCols ? s_ref[gt] : 0.0f;  // of row gt, before the next piece's
      column_sums(sum);
      if (!(lane & 1)) s_red[gw * kCols + (lane >> 1)] = sum[0];
      have = !any(!ok || next.cnt == 0);
      if (M::kQs == 1 && have) prepare(next, p + 1);
      float l = 0.0f;  // row gt's sum, and reference
      float ref = mine_ref;
      if (gt < kCols) {
        l = (s_red[gt] + s_red[16 + gt]) + (s_red[32 + gt] + s_red[48 + gt]);
        if (kTurns == 1) {
          s_fac[gt] = l == 0.0f ? 0.0f : 1.0f / l;  // 0: a row that sees nothing
        } else {  // for the other group: in the place of the warps' sums, which this thread alone reads
          s_red[gt] = ref;
          s_red[16 + gt] = l;
        }
      }
      if (ok) ok = bar_wait(o_full, (uint32_t)p & 1u);
      fence_after();
      const bool mine = D == 128 || gw < 2;
      const int d = gt;
      float o[kCols];
      {
        float rest[kCols];
        tmem_ld16(tmem + lanes + o_at + n0, o);
        tmem_ld16(tmem + lanes + o_at + N + n0, rest);
        tmem_ld_wait(o);
        tmem_ld_wait(rest);
#pragma unroll
        for (int n = 0; n < kCols; ++n) o[n] = kF8 ? o[n] + rest[n] : add_low(o[n], rest[n]);
        if (kF8) {
          tmem_ld16(tmem + lanes + o_at + 2 * N + n0, rest);
          tmem_ld_wait(rest);
#pragma unroll
          for (int n = 0; n < kCols; ++n) o[n] = fmaf(rest[n], 0.00390625f, o[n]);
          tmem_ld16(tmem + lanes + o_at + 3 * N + n0, rest);
          tmem_ld_wait(rest);
#pragma unroll
          for (int n = 0; n < kCols; ++n) o[n] = fmaf(rest[n], 0.00390625f, o[n]) * 0.0078125f;  // 2^-7
        }
      }
      // the values that left the products, to the rows that see them: once a piece, after its groups' sums are
      // over one reference (0 times an infinity is NaN)
      auto add_odd = [&]() {
        if (kF8 || !ms.odd[p & 3]) return;
#pragma unroll 1
        for (int k = 0; k < 4 && mine; ++k) {
          if (!((ms.odd[p & 3] >> k) & 1)) continue;
          const int k0 = (cur.tile0 + (k < 2 ? k : cur.tiles - 1 - (k - 2))) * kTile;
#pragma unroll 1
          for (int key = k0; key < min(k0 + kTile, tokens); ++key) {
            const int pg = page_of(a, key), page = table[pg];
            if (page < 0 || page >= a.c.pages || sees(every, key, cur.len)) continue;
            const float v = bf16_bits_to_f32(
                ((const uint16_t*)a.c.v)[page * a.c.page_stride + (key - pg * ps) * a.c.token_stride +
                                         cur.h * a.c.head_stride + d]);
            if (finite_(v)) continue;
#pragma unroll
            for (int n = 0; n < kCols; ++n)
              if (sees(rows_of(p)[n0 + n], key, cur.len)) o[n] += v;
          }
        }
      };
      fence_before();
      bar_arrive(o_empty);
      if (kTurns > 1) {
        // both groups' sums over one reference; the first adds the second's
        warps_sync<kBoth>(kBothId);
        const float* other = s_red + (turn == 0 ? 4 : -4) * kCols;
        const bool any_mine = i0 < cur.cnt;  // else nothing of this piece is in its accumulators
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          const float f = exp2_(s_red[n] - fmaxf(s_red[n], other[n]));
          o[n] = any_mine ? o[n] * f : 0.0f;
        }
        float* sums = reinterpret_cast<float*>(sm + M::kP + M::kPlace);  // [16][D], where its weights were
        if (turn > 0) {
          if (mine) {
#pragma unroll
            for (int n = 0; n < kCols; ++n) sums[n * D + d] = o[n];
          }
          warps_sync<kBoth>(kBothId);
          continue;
        }
        if (gt < kCols) {
          const float top = fmaxf(ref, other[gt]);
          l = l * exp2_(ref - top) + other[16 + gt] * exp2_(other[gt] - top);
          ref = top;
          s_fac[gt] = l == 0.0f ? 0.0f : 1.0f / l;
        }
        warps_sync<kBoth>(kBothId);
        if (mine) {
#pragma unroll
          for (int n = 0; n < kCols; ++n) o[n] += sums[n * D + d];
        }
        if (have) warps_arrive<kBoth>(kSumId);
      } else {
        warps_sync<kGroup>(bid);  // s_fac
      }
      add_odd();
      const bool whole = cur.cnt == cur.tiles;
      const int64_t slot = (int64_t)(2 * blockIdx.x + (cur.first == 0 ? 1 : 0)) * N;
      auto put_lse = [&](int n, float ref, float l) {
        const int v = cur.h0 + n, j = v / a.group;
        if (a.lse)
          a.lse[(int64_t)(cur.row0 + cur.j0 + j) * a.q_heads + cur.h * a.group + v - j * a.group] =
              l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
      };
      // Small units are often nearly empty (a row a head): a thread puts its column where its rows' weights were,
      // and a short loop takes the rows there are (70 requests of 32 heads 171 us, all 16 written out, and 152 so;
      // verify windows 72 and 69; 32 rows in E4M3 35 and 38, 64 rows 43 and 45: those write out all)
      constexpr bool kShort = N == 16 || (N == 32 && !kF8);
      const int rows_here = min(kCols, cur.valid - n0);
      auto column = [&](int n) {
        unsigned char* at = kF8 ? s_p + (n >> 2) * (kTile * 16) + (n & 3) * (D * 4)
                                : s_p + (n0 >> 3) * (kTile * 16) + (n >> 3) * (2 * N * kTile) + (n & 7) * (D * 4);
        return reinterpret_cast<float*>(at) + d;
      };
      if (kShort && mine) {
#pragma unroll
        for (int n = 0; n < kCols; ++n) *column(n) = o[n];
      }
      if (whole) {
        if (mine) {
          int j = (cur.h0 + n0) / a.group, hq = cur.h0 + n0 - j * a.group;
          uint16_t* to = a.out + (cur.row0 + cur.j0 + j) * a.ldo + (int64_t)(cur.h * a.group + hq) * D + d;
          auto put = [&](int n, float x) {
            const float inv = s_fac[n];
            *to = f32_to_bf16_bits(inv == 0.0f ? 0.0f : x * inv);
            to += D;
            if (++hq == a.group) hq = 0, to += a.ldo - (int64_t)a.group * D;
          };
          if (kShort) {
#pragma unroll 1
            for (int n = 0; n < rows_here; ++n) put(n, *column(n));
          } else {
#pragma unroll
            for (int n = 0; n < kCols; ++n)
              if (n < rows_here) put(n, o[n]);
          }
        }
        if (gt < kCols && n0 + gt < cur.valid) put_lse(n0 + gt, ref, l);
      } else {
        const int b0 = (int)cuts.owner(cur.line0, cur.tiles), pieces = (int)cuts.pieces(cur.line0, cur.tiles);
        if (kShort) {
#pragma unroll 1
          for (int n = 0; n < rows_here && mine; ++n) __stcg(a.acc + (slot + n0 + n) * D + d, *column(n));
        } else {
#pragma unroll
          for (int n = 0; n < kCols; ++n)
            if (n < rows_here && mine) __stcg(a.acc + (slot + n0 + n) * D + d, o[n]);
        }
        if (gt < kCols && n0 + gt < cur.valid) __stcg(a.ml + slot + n0 + gt, make_float2(ref, l));
        warps_sync<kGroup>(bid);
        if (gt == 0) {
          __threadfence();
          int32_t* count = a.count + b0 * R::kGroups + grp;
          const int was = atomicAdd(count, 1);
          ms.last[grp] = was == pieces - 1;
          if (ms.last[grp]) *count = 0;
        }
        warps_sync<kGroup>(bid);
        if (ms.last[grp]) {  // all pieces are there: added in their order
          __threadfence();
          auto slot_of = [&](int k) { return (int64_t)(k == 0 ? 2 * b0 + 1 : 2 * (b0 + k)) * N + n0; };
          const int mine_n = min(kCols, cur.valid - n0);
          // each row's reference and sum: 8 threads a row, a piece in turn
          const int jn = gt & 15;
          auto stat = [&](int k) {
            return k < pieces && jn < mine_n ? __ldcg(a.ml + slot_of(k) + jn) : make_float2(kUnset, 0.0f);
          };
          const float2 own = stat(gt / 16);
          float top = own.x;
#pragma unroll 1
          for (int k = gt / 16 + 8; k < pieces; k += 8) top = fmaxf(top, stat(k).x);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          if (lane < 16) s_red[gw * 16 + jn] = top;
          warps_sync<kGroup>(bid);
          top = fmaxf(fmaxf(s_red[jn], s_red[16 + jn]), fmaxf(s_red[32 + jn], s_red[48 + jn]));
          // E4M3: references hold the values' scales, so that of a piece with few of the weights can be far above
          // that of one with many
          auto over_top = [&](const float2& st) {
            return kF8 ? lowered(st.y, st.x - top) : exp2_(st.x - top) * st.y;
          };
          float sums = over_top(own);
#pragma unroll 1
          for (int k = gt / 16 + 8; k < pieces; k += 8) sums += over_top(stat(k));
          sums += __shfl_xor_sync(0xffffffffu, sums, 16);
          warps_sync<kGroup>(bid);
          if (lane < 16) s_red[gw * 16 + jn] = sums;
          warps_sync<kGroup>(bid);
          sums = (s_red[jn] + s_red[16 + jn]) + (s_red[32 + jn] + s_red[48 + jn]);
          if (gt < kCols) {
            s_ref[gt] = top;  // the next piece's is set after
            s_fac[gt] = sums == 0.0f ? 0.0f : 1.0f / sums;
            if (gt < mine_n) put_lse(n0 + gt, top, sums);
          }
          warps_sync<kGroup>(bid);
          // several rows a thread at once, 4 dims of each
          constexpr int T = D / 4, kRowsAt = kGroup / T, kEach = kCols / kRowsAt;
          constexpr int kBatch = (N == 64 ? 8 : 16) / kEach;  // pieces read at once
          const int d4 = gt % T * 4, r0 = gt / T;
          float4 v[kEach];
          float tops[kEach];
#pragma unroll
          for (int u = 0; u < kEach; ++u) {
            v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            tops[u] = s_ref[r0 + u * kRowsAt];
          }
          // many pieces are read several at once (one row over 55000 tokens 38 us, one by one, and 31 so); for few
          // the longer loop's instructions take longer to come than its reads (E4M3 batch 127 us and 132)
          if (pieces <= 4) {
#pragma unroll 1
            for (int k = 0; k < pieces; ++k)
#pragma unroll
              for (int u = 0; u < kEach; ++u) {
                const int n = r0 + u * kRowsAt;
                if (n < mine_n) {
                  const float f = exp2_(__ldcg(a.ml + slot_of(k) + n).x - tops[u]);
                  const float4 x = __ldcg(reinterpret_cast<const float4*>(a.acc + (slot_of(k) + n) * D + d4));
                  v[u].x += f * x.x, v[u].y += f * x.y, v[u].z += f * x.z, v[u].w += f * x.w;
                }
              }
          } else {
#pragma unroll 1
            for (int k0 = 0; k0 < pieces; k0 += kBatch) {
              float f[kBatch][kEach];
              float4 x[kBatch][kEach];
#pragma unroll
              for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int u = 0; u < kEach; ++u) {
                  const int n = r0 + u * kRowsAt;
                  const bool in = k0 + k < pieces && n < mine_n;
                  f[k][u] = in ? __ldcg(a.ml + slot_of(k0 + k) + n).x : -INFINITY;
                  x[k][u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                  if (in) x[k][u] = __ldcg(reinterpret_cast<const float4*>(a.acc + (slot_of(k0 + k) + n) * D + d4));
                }
#pragma unroll
              for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int u = 0; u < kEach; ++u) {
                  const float e = exp2_(f[k][u] - tops[u]);
                  v[u].x += e * x[k][u].x, v[u].y += e * x[k][u].y;
                  v[u].z += e * x[k][u].z, v[u].w += e * x[k][u].w;
                }
            }
          }
#pragma unroll
          for (int u = 0; u < kEach; ++u) {
            const int n = r0 + u * kRowsAt;
            if (n >= mine_n) continue;
            const float inv = s_fac[n];
            const int r = cur.h0 + n0 + n, j = r / a.group;
            uint2 w = make_uint2(bf16x2(v[u].x * inv, v[u].y * inv), bf16x2(v[u].z * inv, v[u].w * inv));
            if (inv == 0.0f) w = make_uint2(0u, 0u);
            *reinterpret_cast<uint2*>(a.out + (cur.row0 + cur.j0 + j) * a.ldo +
                                      (int64_t)(cur.h * a.group + r - j * a.group) * D + d4) = w;
          }
        }
      }
    }
  }
  if (!ok) set_dev_status(a.dev_status, TFD_ERR_TIMEOUT);
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == kScoreWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem)
                 : "memory");
}

// Rows of a unit: 16 where a request's rows of a key head fit, else 32, or 64 (bf16; E4M3's four parts a row fill
// tensor memory at 32) where a head has several units of 64, which then read its tokens half as often, and such
// units are there for half the SMs: 48 requests of 32 rows, 8 query heads a key head, 1034 us and with 32 1202; four
// such of few tokens 22 and 15, one unit of 40 rows 23 and 14.
inline int unit_rows(int rows, int fmt, int64_t heads, int sms) {
  if (rows <= 16) return 16;
  return fmt == TFD_KV_BF16 && rows > 64 && heads * ((rows + 63) / 64) >= sms / 2 ? 64 : 32;
}

inline size_t workspace(int rows_of_unit, int dim) {
  const size_t rows = (size_t)2 * kMaxBlocks * rows_of_unit;
  return kMaxBlocks * 16 + rows * 8 + rows * dim * 4;
}

template <int D, int N, bool kF8>
tfd_status launch(const Args<D>& a, cudaStream_t stream) {
  int dev = 0;
  const int sms = tfd_host::device_sms(dev);
  constexpr int smem = Smem<D, N, kF8>::kBytes;
  return tfd_host::launch_clusters<paged_attn_kernel<D, N, kF8>>(
      a, dev, std::min(kMaxBlocks, std::max(1, sms * Roles<D, N, kF8>::kCtas)), 1, Roles<D, N, kF8>::kT, smem, smem,
      stream);
}

template <int D>
tfd_status launch_dim(Args<D>& a, float rope_base, cudaStream_t stream) {
  a.page_stride = (int)a.c.page_stride, a.token_stride = (int)a.c.token_stride;
  a.head_stride = (int)a.c.head_stride;
  if (a.qk & TFD_QK_ROPE) a.turns = tfd_host::rope_turns<D>(rope_base);
  int dev = 0;
  const int n = unit_rows(a.max_new * a.group, a.c.fmt, (int64_t)a.requests * a.c.heads, tfd_host::device_sms(dev));
  if (a.c.fmt == TFD_KV_E4M3)
    return n == 16 ? launch<D, 16, true>(a, stream) : launch<D, 32, true>(a, stream);
  return n == 16   ? launch<D, 16, false>(a, stream)
         : n == 32 ? launch<D, 32, false>(a, stream)
                   : launch<D, 64, false>(a, stream);
}

}  // namespace

extern "C" size_t tfd_paged_attn_workspace(int max_new, int q_heads, int heads, int dim) {
  if (max_new < 1 || max_new > TFD_MAX_ROWS || heads < 1 || heads > 1024 || q_heads < heads ||
      q_heads % heads || q_heads / heads > 64 || (dim != 64 && dim != 128))
    return 0;
  return workspace(unit_rows(max_new * (q_heads / heads), TFD_KV_BF16, 1, 0), dim);
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
      ldt > ((int64_t)1 << 40) || (int64_t)rows * q_heads > 2147483647 ||
      std::max({c.page_stride, c.token_stride, c.head_stride}) > 2147483647)
    return TFD_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(row_start, 4) || !aligned(pos, 4) || !aligned(tree, 4) || !aligned(q_gamma, 2) ||
      !aligned(lse, 4) || !aligned(dev_status, 4) || !aligned(ws, 16))
    return TFD_ERR_INVALID;
  const int group = q_heads / c.heads;
  const int most_rows = unit_rows(max_new * group, TFD_KV_BF16, 1, 0);  // of a unit, whatever the form
  const size_t need = workspace(most_rows, c.dim);
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
  const size_t slots = (size_t)2 * kMaxBlocks * most_rows;
  int32_t* count = (int32_t*)w;
  float2* ml = (float2*)(w + kMaxBlocks * 16);
  float* acc = (float*)(w + kMaxBlocks * 16 + slots * 8);
  cudaStream_t s = tfd_host::as_stream(stream);
  // 2^(31 + b) / page_size rounded up, b the bits of page_size - 1: exact for tokens below 2^31
  uint32_t shift = 0;
  while ((1 << shift) < c.page_size) ++shift;
  const uint32_t mul = (uint32_t)((((uint64_t)1 << (31 + shift)) + c.page_size - 1) / c.page_size);
#define TFD_ATTN_DIM(D)                                                                          \
  if (c.dim == D) {                                                                              \
    Args<D> a = {(const uint16_t*)q, ldq, table, ldt, lens, row_start, pos, tree,                \
                 (const uint16_t*)q_gamma, (uint16_t*)out, ldo, lse, count, ml, acc, dev_status, \
                 c, rows, q_heads, group, max_pages, requests, max_new, window, qk, eps, sc,     \
                 mul, shift};                                                                    \
    return launch_dim<D>(a, rope_base, s);                                                       \
  }
  TFD_ATTN_DIM(64)
  TFD_ATTN_DIM(128)
#undef TFD_ATTN_DIM
  return TFD_ERR_UNSUPPORTED;
}
