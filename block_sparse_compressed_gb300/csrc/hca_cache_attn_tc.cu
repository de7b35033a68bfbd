// hca_cache_attn_tc.cu -- attention over the 8-bit cache on the tensor cores
// (tcgen05 + TMEM), bf16 queries, D = 64 or 128.
//
// A CTA takes a range of the line of tiles (hca_cache.cuh).  A tile is 128 keys
// of one group, a group NQ (position, head) rows of a request:
//   S [128 x 128 keys]  = Q [128 x D] K^T       kind::f16, Q and K from shared memory
//   O [128 x D]        += P [128 x 128 keys] K   kind::f16, P from tensor memory
// With the rows in the lanes of tensor memory a softmax thread owns a row: its
// maximum and its sum stay in its registers and nothing is exchanged between
// threads.  (Keys in the lanes instead waste none of the M dimension on a single
// token's 64 heads and can use the e4m3 rows as they are, but every maximum then
// crosses 128 threads: 4,200 cycles a tile were measured, half of them there.)
//
// A tile goes in two halves of 64 keys: while the softmax works on one, the
// tensor cores add the other's part of O and make its next scores.
//
// The products take 128 rows whatever NQ is, so a group of NQ = 64 (32) rows has
// them in the lanes twice (four times), and each copy sees its own half
// (quarter) of a half's keys: P is zero for the others.  The copies are so many
// independent streams of the online softmax, joined when the group ends.
//
// The cache's e4m3 values become fp16 once for both products and all rows.  A page
// is contiguous, so one bulk copy brings it to shared memory, into the half of its
// fp16 rows' bytes that the converter warps overwrite last; they also make q ready
// (below) while the softmax warps end the group before.  q becomes fp16 with a
// power of two for each row that puts its largest value at 224 .. 448: bf16's 8
// bits fit, what falls below 2^-14 loses bits (2^-33 of the row's largest value).
//
// Block scales go into the keys: a page of scale s is stored as k8 * 2^e in units
// of 2^u, with s = 2^(u + e) and u the same for all of a segment's tiles, which
// fp16 holds exactly for e in -15 .. 7.  So scores need one factor for all keys,
// and the probabilities, rounded to fp16 (11 bits; 2^-25 of the row's reference
// where tiny), and their sum do not depend on scales.  (p * s rounded to fp16
// loses every key but those of the blocks with the largest scales, whatever their
// values are, and a sum of (p * s) / s leaves fp32's range with s.)  u is the
// largest scale of the segment's first tile; a page more than 2^7 beyond it raises
// u, and O follows.  What is left of a scale below 2^-15 of the unit, or of one that
// is no power of two, multiplies its scores and probabilities in tensor memory, in
// functions of their own that ordinary tiles only pass by.  The factors take the
// converter 3 of 95 us at m = 4.  (Other ways, there and for prompts of 2,571 tokens,
// where this one took 93.4 and 74.0: scales for every 16 keys in the softmax 96.5
// and 78.0, the rest beside them 96.9 and 83.5; a unit for each half and a second
// loop for those that need factors 93.8 and 79.2.)
//
// The reference exponent of a row is 2 below its largest score so far, so that fp16
// reaches down to 2^-27 of the largest probability, and raised only when that score
// is beaten by 2^11, so that O is rarely rescaled: a row of a warp that needs it
// costs all 32 a trip through O.  (64 tokens at m = 4 and prompts of 2,571 tokens,
// 6 and 7 instead: 95.9 and 76.5 us; 4 and 9: 95.2 and 75.8; 2 and 11: 94.3 and 75.4;
// 0 and 13: 93.6 and 75.2.)  fp16 ends at 2^16: scores of 2^24 are 1.44 * 2^24 in
// base 2, where fp32 has steps of 2, and the roundings of the score, the threshold
// and the reference add at most 2 to those 13.
//
// A row of the cache that some query row does not see may hold anything, and
// 0 * NaN is not 0: of the pages that not every row sees whole, the converter
// stores zeros for keys with a NaN and notes them in a bit mask, by which the
// softmax gives a NaN to whoever sees them.
//
// Bounds.  A half's scores take the tensor cores 384 cycles (8 products of 128 x
// 64 x 16 at 48, bound by their operands from shared memory) and its part of O
// 254, so a tile 1,228 when products are queued; but the time from issue to the
// softmax's first look is 805 and 590, and a half's softmax about 1,100.  Two CTAs
// of an SM fill part of each other's gaps: 64 tokens over 95,000 rows each (199 MB
// of cache, 64 heads, D = 128) take 95.5 us, 2.1 TB/s and 529 TFLOP/s, with the
// tensor cores busy half of the time (timing copies of a build of 94.8 us: 81.6 with
// one product of each half left, 87.3 with half of the score products, 93 with half
// of the output products or without exponentials, 91.5 without the keys' factors).
// One decode step of 64 requests at 128
// keys an entry takes 22.5 us: the schedule, the way to the first scores and the way
// out are most of it.  Chunks of 2,571 prompt tokens take 75.0 us, 67.9 with one
// product left: beginnings and ends of their groups of 2 tokens.
// Measured and left, each against the kernel of its time: scores of a whole tile
// at once (128 x 128 x 16 at 64 cycles: the tensor cores do less, but the softmax
// waits: 109 us for 102); two softmax warpgroups, a half each (99 us for 96: the
// products' latency is the limit, not the softmax's); pages through the
// converter's registers (the same time, 4 KB more code); the next tile's loads
// between a tile's stores (135 us for 105).
#include <cuda_bf16.h>

#include <cfloat>
#include <climits>
#include <type_traits>

#include "hca_cache_attn.cuh"
#include "tc_tiles.cuh"

namespace hca {
using namespace tc;
using namespace cache;

namespace {

constexpr float kRaiseLog2 = 11.f, kBias = 2.f;
constexpr int kLeastExp = -15, kMostExp = 7;      // e: 2^-9 .. 448 times 2^e is an fp16 value
constexpr int kLeastUnit = -100, kMostUnit = 127;  // u: 2^u / l is a normal number (l below 2^26)
constexpr int kLeastQExp = -118;                  // exponent of q's factor: so is its reciprocal
constexpr int kMetaStages = 4;  // tiles whose pages are looked up ahead
constexpr int kStages = 2;      // fp16 tiles; filled and released by halves
constexpr int kHalfStages = 2 * kStages;
constexpr int kMaxSegs = 64;    // pieces of groups listed in shared memory
constexpr int kWG = 128;
constexpr int kThreads = 3 * kWG;  // softmax | converter | page, MMA and copy warps
constexpr int kTmem = 256;      // S of keys 0 .. 63 | S of keys 64 .. 127 (P takes the first half of each) | O
constexpr uint32_t kColO = 128;
enum { kBarOut = 1, kBarQ = 2 };  // named barriers of the softmax's and the converter's warps

template <int NQ, int D>
struct Cfg {
  static constexpr int kCopies = 128 / NQ;                 // of a row in the lanes
  // Registers: 2 CTAs of 384 threads leave 80 each; a softmax thread holds kSpan scores.
  static constexpr int kRegsSoft = 128, kRegsConv = 56, kRegsIssue = 56;
  static_assert(kRegsSoft + kRegsConv + kRegsIssue <= 3 * 80, "register split must fit the launch");
  static constexpr int kSpan = 64 / kCopies;               // keys of a half that a thread takes: 64, 32, 16
  static constexpr int kHalves = D / 64;                   // 128-byte column blocks of an fp16 row
  static constexpr int kStageBytes = kHalves * kHalfTile;  // fp16 tile of 128 keys
  static constexpr int kOffQ = kStages * kStageBytes;
  // e4m3 rows as they are in the cache: of 128 bytes in the columns 64 .. 127 of
  // their fp16 rows, of 64 bytes behind q
  static constexpr int kOffRaw = D == 128 ? kHalfTile : kOffQ + kHalves * kHalfTile;
  static constexpr int kRawStride = D == 128 ? kStageBytes : kTileKeys * D;
  static constexpr int kSmem = kOffQ + kHalves * kHalfTile + (D == 128 ? 0 : kStages * kRawStride) + 1024;
};

enum PageKind { kRaw = 0, kComp = 1, kNoPage = 2, kAllSeen = 3 };  // kAllSeen: every row sees every key

struct __align__(16) PageMeta {
  const uint8_t *rows;  // NULL: no page, or a bad block id
  int key0, kind;
  float rest;           // the page's scale is 2^(unit + e) * rest
  uint32_t factor;      // 2^e, for both values of a pair of fp16
  int pad[2];
};

template <int NQ, int D>
struct Shared {
  uint4 join[kWG * 4];  // O on its way out: 64 bytes of each lane's row
  uint64_t meta_full[kMetaStages], meta_empty[kMetaStages];
  uint64_t raw_full[kHalfStages], kv_full[kHalfStages], kv_empty[kHalfStages];
  uint64_t q_full, q_read, s_full[2], p_full[2], pv_done[2], drain, never;
  PageMeta meta[kMetaStages][8];
  uint32_t nan_keys[kMetaStages][4];  // keys whose rows hold a NaN that not everybody sees
  int nan_any[kMetaStages];
  int all_seen[kMetaStages];          // bit h: every row sees every key of half h
  uint32_t valid[kMetaStages];        // bit i: there is a page i
  int unit[kMetaStages];              // exponent of the tile's keys in fp16
  // hardly ever not 0: (the unit of the tile in front less this one's) * 2 + (a
  // page's rest is not 1)
  int odd[kMetaStages];
  // the CTA's pieces of groups, in order; what there is no room for is in the
  // workspace's groups
  Segment seg[kMaxSegs];
  int gbase[kThreads];
  float q_factor[NQ];                            // log2(e) |scale| / (a row's factor)
  float2 ml[kWG];                                // copies: reference and sum of every lane
  int2 sums[2][kThreads / 32];                   // tiles and groups of each warp
  uint32_t tmem_base;
  int abort, first, range[2];
};

// s = 2^exponent * part with part in (0.5, 1], for positive finite s.
__device__ __forceinline__ int split_scale(float s, float &part) {
  const int sub = s < FLT_MIN ? 24 : 0;  // a subnormal one
  const uint32_t u = __float_as_uint(sub ? s * 16777216.f : s), mant = u & 0x7fffffu;
  part = mant ? __uint_as_float(mant | (126u << 23)) : 1.f;
  return (int)(u >> 23) - (mant ? 126 : 127) - sub;
}
// 2^e in both halves, e in [kLeastExp, kMostExp]
__device__ __forceinline__ uint32_t f16x2_exp2(int e) { return (e >= -14 ? (uint32_t)(e + 15) << 10 : 0x400u >> (-14 - e)) * 0x10001u; }
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void ld_shared(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 16 bytes of which the first n come from p and the others are 0
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *p, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
               "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// 4 e4m3 values -> two fp16 pairs
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t &a, uint32_t &b) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(w));
}

// Sum of v over the threads in front of this one, total and number of those
// that count; a warp's v sum up to less than 2^31 (a group has 2^25 tiles at
// most).
static __device__ __noinline__ int scan_tiles(int v, bool counts, int2 *sums, long long &total, int &ncounts, int &index) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  const uint32_t b = __ballot_sync(0xffffffffu, counts);
  if (lane == 31) sums[warp] = make_int2(x, __popc(b));
  __syncthreads();
  int before = x - v, n = 0, idx = __popc(b & ((1u << lane) - 1u));
  long long all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int2 s = sums[w];
    if (w < warp) before += s.x, idx += s.y;
    all += s.x;
    n += s.y;
  }
  total = all;
  ncounts = n;
  index = idx;
  return before;
}

// Scores of kSpan keys from column k0 of a tile on, times their pages' rests.
template <int kSpan>
static __device__ __noinline__ void scale_s(uint32_t addr, const PageMeta *meta, int k0, int log_bs) {
#pragma unroll 1
  for (int c = 0; c < kSpan; c += 16) {
    const float rest = meta[(k0 + c) >> log_bs].rest;
    uint32_t v[16];
    tmem_ld16(addr + c, v);
    tmem_wait_ld();
#pragma unroll
    for (int y = 0; y < 16; ++y) v[y] = __float_as_uint(__uint_as_float(v[y]) * rest);
    tmem_st16(addr + c, v);
  }
  tmem_wait_st();
}

// Probabilities of kSpan keys whose scores lie at `s`, times their pages' rests, to
// `to` (which a key's score has left by then); returns the sum of the
// probabilities themselves.
template <int kSpan>
static __device__ __noinline__ float scaled_p(uint32_t s, uint32_t to, float ck, float m_use, const PageMeta *meta, int k0, int log_bs) {
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < kSpan; c += 16) {
    const float rest = meta[(k0 + c) >> log_bs].rest;
    uint32_t v[16], pk[8];
    tmem_ld16(s + c, v);
    tmem_wait_ld();
#pragma unroll
    for (int y = 0; y < 16; y += 2) {
      const float e0 = ex2_approx(fmaf(__uint_as_float(v[y]), ck, -m_use)), e1 = ex2_approx(fmaf(__uint_as_float(v[y + 1]), ck, -m_use));
      sum += e0 + e1;
      pk[y >> 1] = f16x2_rn(e0 * rest, e1 * rest);
    }
    tmem_st8(to + c / 2, pk);
  }
  tmem_wait_st();
  return sum;
}

// A warp's rows of O times f.
template <int D>
static __device__ __noinline__ void scale_o(uint32_t addr, float f) {
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t o[16];
    tmem_ld16(addr + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
    tmem_st16(addr + c, o);
  }
  tmem_wait_st();
}

template <int NQ, int D>
__global__ void __launch_bounds__(kThreads, 2) hca_cache_attn_kernel(const AttnParams p) {
  using C = Cfg<NQ, D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Shared<NQ, D> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int *abort_flag = &sh.abort;
  int32_t *status = &p.err[blockIdx.x];

  if (tid == 0) {
#pragma unroll 1
    for (int s = 0; s < kMetaStages; ++s) {
      mbar_init(&sh.meta_full[s], 1);
      mbar_init(&sh.meta_empty[s], kWG);  // the softmax is the last to read a tile's pages
    }
#pragma unroll 1
    for (int s = 0; s < kHalfStages; ++s) {
      mbar_init(&sh.raw_full[s], 1);
      mbar_init(&sh.kv_full[s], kWG);
      mbar_init(&sh.kv_empty[s], 1);
    }
    mbar_init(&sh.q_full, kWG);
    mbar_init(&sh.q_read, kWG);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&sh.s_full[h], 1);
      mbar_init(&sh.p_full[h], kWG);
      mbar_init(&sh.pv_done[h], 1);
    }
    mbar_init(&sh.drain, 1);
    mbar_init(&sh.never, 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 10) {
    tmem_alloc(&sh.tmem_base, kTmem);
    tmem_relinquish();
  }
  // the CTA's range of the line, and its pieces of groups
  int ntiles, quota, c0 = 0, c1 = 0;
  bool busy = false;
  if (p.in_cta) {
    // one thread per request; where some bring more than one group, one per group
    int n = 0, r = tid, k = 0;
    bool ok = true;
    if (tid < p.R) ok = request_chunks(p, tid, n);
    bool mine = n == 1;
    if (__syncthreads_or(n > 1)) {
      long long all;
      int unused;
      const int chunks = scan_tiles(n, false, sh.sums[1], all, unused, unused);
      if (tid < p.R) sh.gbase[tid] = chunks;
      __syncthreads();
      mine = tid < all;
      int hi = p.R;  // gbase[r] <= tid < gbase[hi]
#pragma unroll 1
      for (r = 0; hi - r > 1;) {
        const int mid = (r + hi) >> 1;
        if (sh.gbase[mid] <= tid) r = mid; else hi = mid;
      }
      k = tid - sh.gbase[r];
    }
    ok = __syncthreads_and(ok);
    Group g;
    g.ntiles = 0;
    mine = mine && ok;
    if (mine) ok = chunk_group(p, r, k, g);
    int ngroups, index;
    long long total;
    g.tile0 = scan_tiles(mine ? g.ntiles : 0, mine, sh.sums[0], total, ngroups, index);
    ntiles = __syncthreads_and(ok) && total < kMaxTiles ? (int)total : -1;
    // Ranges that no group's border cuts give a CTA tiles of one group only and
    // save it a second one's beginning and end, about two tiles' time each;
    // ceil(tiles / quota) of them for each group fit the grid with a larger quota.
    // Up to 2 tiles more they pay: 64 requests over up to 131,072 rows at m = 128 22.6
    // us, 24.9 cut anywhere, 20 over up to 20,000 at m = 4 27.4 and 30.7; more do not:
    // 140 over 3,000 rows 24.8 cut anywhere, 30.8 with 4 more, 64 over 60,000 to
    // 131,072 rows 95 cut anywhere, 107 with as many as it takes.
    quota = cta_quota(ntiles, p.grid, p.min_tiles);
    const int own = cta_quota(ntiles, max(p.grid - ngroups, 1), p.min_tiles);
    const bool whole_groups = ngroups < p.grid && own <= quota + 2;
    if (whole_groups) {
      quota = own;
      g.tile0 = quota * scan_tiles(mine ? (g.ntiles + quota - 1) / quota : 0, mine, sh.sums[1], total, ngroups, index);
    }
    c0 = quota * blockIdx.x;
    c1 = whole_groups ? c0 + quota : min(c0 + quota, ntiles);
    const bool in = mine && ntiles > 0 && g.tile0 < c1 && g.tile0 + g.ntiles > c0;
    if (in && g.tile0 <= c0) sh.first = index;
    busy = __syncthreads_or(in);
    if (in) {
      Segment x = segment_of(g, c0, c1, blockIdx.x);
      if (whole_groups) x.slice_last |= 1;
      if (index - sh.first < kMaxSegs) sh.seg[index - sh.first] = x;
      else p.groups[index] = g;
      if (x.last()) p.border[blockIdx.x] = border_of(p, g, c0, c1, quota, blockIdx.x);
    }
  } else {
    pdl_wait();  // for the schedule
    ntiles = p.hdr->ntiles;
    quota = cta_quota(ntiles, p.grid, p.min_tiles);
    busy = ntiles > 0 && blockIdx.x <= (ntiles - 1) / quota;
    const int ng = p.hdr->ngroups;
    // cut between groups: 2 and more for each CTA, short ones, and none of them more
    // than half of a CTA's share
    const long long line = ntiles + (long long)kGroupCost * ng;
    const int share = (int)min((line + p.grid - 1) / p.grid, 0x7fffffffll);
    if (ng >= 2 * p.grid && line < kMaxTiles && p.hdr->longest <= min(kShortGroup, share / 2 - kGroupCost) && ntiles > 0) {
      if (warp < 2) {
        // the first group that begins at or behind the share's beginning (end)
        const long long at = (long long)share * (blockIdx.x + warp);
        const int g = at == 0 ? 0 : at > line ? ng : find_group(p.groups, ng, (int)at - 1, kGroupCost) + 1;
        if (lane == 0) sh.range[warp] = g < ng ? p.groups[g].tile0 : ntiles;
        if (warp == 0 && lane == 0) sh.first = g;
      }
      if (tid == 0) p.border[blockIdx.x] = Border{0, 0, 0, 0};
      __syncthreads();
      c0 = sh.range[0];
      c1 = sh.range[1];
      busy = c0 < c1;
    } else if (busy) {
      c0 = quota * blockIdx.x;
      c1 = min(c0 + quota, ntiles);
      if (warp < 2) {
        const int g = find_group(p.groups, ng, warp ? c1 - 1 : c0);
        if (warp == 0 && lane == 0) sh.first = g;
        if (warp == 1 && lane == 0) p.border[blockIdx.x] = border_of(p, p.groups[g], c0, c1, quota, blockIdx.x);
      }
      __syncthreads();
    }
    if (busy) {
      const int gi = sh.first + tid;
      if (tid < kMaxSegs && gi < ng) {
        const Group g = p.groups[gi];
        if (g.tile0 < c1) sh.seg[tid] = segment_of(g, c0, c1, blockIdx.x);
      }
    }
  }
  if (tid == 0) {
    p.err[blockIdx.x] = ntiles < 0 ? HCA_ERR_CACHE : HCA_OK;
    if (!busy) p.border[blockIdx.x] = Border{0, 0, 0, 0};
  }
  const uint32_t limit_ns = (uint32_t)p.wait_ns;
  auto wait_bar = [&](uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_idle(bar, parity, abort_flag, limit_ns));
  };
  pdl_launch_dependents();  // the combine kernel waits for this one's end by itself
  auto segment = [&](int k) { return k < kMaxSegs ? sh.seg[k] : segment_of(p.groups[sh.first + k], c0, c1, blockIdx.x); };
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  const int ppt = kTileKeys >> p.log_bs;  // pages per tile: a power of two, 1 .. 8
  if (warp >= 8) {
    setmaxnreg_dec<C::kRegsIssue>();
    if (warp == 8 && busy) {
      // ------------------------------------------------------------ pages
      const int batch = 32 / ppt;  // tiles whose pages the warp's lanes look up at once
      const uint32_t page_bytes = D << p.log_bs;
      uint32_t n = 0;
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        int unit = 0;
        bool set = false;  // by the segment's first pages
        const Segment g = segment(k);
        const Pages pg = group_pages(g.pos0, g.npos, p.W, p.m, p.log_bs, p.comp.table != nullptr);
#pragma unroll 1
        for (int jb = g.j0; ok && jb < g.j1; jb += batch) {
          const int v = jb * ppt + lane;
          PageMeta pm = {nullptr, 0, kNoPage, 1.f, f16x2_exp2(0), {0, 0}};
          float scale = 1.f;
          bool bad = false;  // block id out of range
          if (v < pg.nraw + pg.ncomp && v < g.j1 * ppt) {
            const bool comp = v >= pg.nraw;
            const CacheSet &cs = comp ? p.comp : p.raw;
            const int page = comp ? v - pg.nraw : pg.rp0 + v;
            const int id = cs.table[(size_t)g.r * cs.cols + page % cs.cols];
            pm.key0 = page << p.log_bs;
            const long long end = (long long)pm.key0 + (1 << p.log_bs);
            const bool all = comp ? end * p.m <= g.pos0 + 1 : end <= (long long)g.pos0 + 1 && pm.key0 > g.pos0 + g.npos - 1 - p.W;
            pm.kind = all ? kAllSeen : comp ? kComp : kRaw;
            if (id >= 0 && id < cs.nblocks) {
              pm.rows = cs.pool + (size_t)id * page_bytes;
              scale = cs.scale[id];
            } else {
              bad = true;  // every key of it is noted as NaN
            }
          }
          const uint32_t seen = __ballot_sync(0xffffffffu, pm.kind == kAllSeen), valid = __ballot_sync(0xffffffffu, pm.rows != nullptr);
          const uint32_t half = (1u << (ppt > 1 ? ppt / 2 : 1)) - 1u;  // pages of a half (one page has both)
          const int jn = min(batch, g.j1 - jb);
#pragma unroll 1
          for (int t = 0; t < jn; ++t, ++n) {
            const int ms = n % kMetaStages;
            if (n >= (uint32_t)kMetaStages)
              ok = wait_bar(&sh.meta_empty[ms], ((n / kMetaStages) - 1) & 1);
            if (!ok) break;
            const bool here = lane / ppt == t;
            PageMeta &to = sh.meta[ms][lane % ppt];
            if (here) {
              if (pm.rows) prefetch_l2(pm.rows, page_bytes);
              to.rows = pm.rows;
              to.key0 = pm.key0;
              to.kind = pm.kind;
            }
            if (lane < 4) sh.nan_keys[ms][lane] = 0;
            if (lane == 0) {
              const uint32_t a = seen >> (t * ppt), b = ppt > 1 ? a >> (ppt / 2) : a;
              sh.nan_any[ms] = 0;
              sh.valid[ms] = (valid >> (t * ppt)) & ((1u << ppt) - 1u);
              sh.all_seen[ms] = ((a & half) == half ? 1 : 0) | ((b & half) == half ? 2 : 0);
            }
            __syncwarp();
            const bool fine = !bad && scale > 0.f && scale < INFINITY;
            float part = 1.f;
            const int ex = here && pm.rows && fine ? split_scale(scale, part) : INT_MIN;
            const int top = __reduce_max_sync(0xffffffffu, ex), was = unit;
            if (top != INT_MIN && (!set || top > unit + kMostExp)) {
              unit = min(max(top, kLeastUnit), kMostUnit);
              set = true;
            }
            const int shift = jb + t == g.j0 ? 0 : max(was - unit, -126);
            if (here) {
              if (!fine) {
                atomicExch(status, HCA_ERR_CACHE);
#pragma unroll 1
                for (int r = (lane % ppt) << p.log_bs, i = 0; i < 1 << p.log_bs; ++i, ++r)
                  atomicOr(&sh.nan_keys[ms][r >> 5], 1u << (r & 31));
                sh.nan_any[ms] = 1;
              }
              if (ex != INT_MIN) {
                const int e = min(max(ex - unit, kLeastExp), kMostExp);
                pm.factor = f16x2_exp2(e);
                pm.rest = part * exp2_int(max(ex - unit - e, -120));
              }
              to.factor = pm.factor;
              to.rest = pm.rest;
            }
            const bool rests = __any_sync(0xffffffffu, here && pm.rest != 1.f);
            if (lane == 0) {
              sh.unit[ms] = unit;
              sh.odd[ms] = 2 * shift + (rests ? 1 : 0);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.meta_full[ms]);
          }
        }
        if (!g.last() && lane == 0) {
          // the next group's rows of q
          const Segment gn = segment(k + 1);
          prefetch_l2(static_cast<const __nv_bfloat16 *>(p.q) + ((size_t)gn.row0 * p.H + gn.slice() * p.HS) * D,
                      real_columns(p, gn.npos, gn.slice()) * D * 2);
        }
        if (g.last()) break;
      }
    } else if (warp == 9 && busy) {
      // ------------------------------------------------------------ MMA
      // One thread's products run in order: S of half (n + 1, h) is issued right
      // behind the O product of (n, h), whose P it overwrites.
      const uint32_t kv0 = smem_u32(smem), q0 = smem_u32(smem + C::kOffQ);
      const uint64_t dk = smem_desc_sw128(kv0, 16, 1024);        // K view of stage 0
      const uint64_t dv = smem_desc_sw128(kv0, kHalfTile, 1024);  // V view of stage 0
      const uint64_t dq = smem_desc_sw128(q0, 16, 1024);
      const uint32_t id_s = idesc_f16_f32(128, 64, false, false), id_o = idesc_f16_f32(128, D, false, true);
      uint32_t n = 0, nseg = 0;
      bool ok = true, issued = false;
      if (p.stall) {
        injected_stall(&sh.never, abort_flag, status, p.wait_ns);
        ok = false;
      }
#pragma unroll 1
      for (; ok; ++nseg) {
        const Segment seg = segment(nseg);
        const int halves = 2 * (seg.j1 - seg.j0);
#pragma unroll 1
        for (int u = 0; ok && u < halves + 2; ++u) {
          const int h = u & 1;
          if (u >= 2) {
            // O of half u - 2
            const uint32_t t = n + (u >> 1) - 1, st = t % kStages;
            ok = wait_bar(&sh.p_full[h], t & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t bv = dv + desc_bytes(st * C::kStageBytes + h * 8192);
            const uint32_t pa = tmem + h * 64, more = u > 2;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mma_ts(tmem + kColO, pa + kk * 8, bv + mnmaj_step(kk), id_o, more || kk > 0);
              mma_commit(&sh.pv_done[h]);
              mma_commit(&sh.kv_empty[2 * st + h]);
            }
            __syncwarp();
          }
          if (u < halves) {
            // S of half u (a group's q is written after the softmax of the group before)
            const uint32_t t = n + (u >> 1), st = t % kStages;
            if (u == 0) ok = wait_bar(&sh.q_full, nseg & 1);
            if (ok) ok = wait_bar(&sh.kv_full[2 * st + h], (t / kStages) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b = dk + desc_bytes(st * C::kStageBytes + h * 8192);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) mma_ss(tmem + h * 64, dq + kmaj_step(kk), b + kmaj_step(kk), id_s, kk > 0);
              mma_commit(&sh.s_full[h]);
            }
            __syncwarp();
            issued = true;
          }
        }
        n += halves / 2;
        if (seg.last()) break;
      }
      if (!ok && issued) {
        volatile int never = 0;
        if (elect_one()) mma_commit(&sh.drain);
        __syncwarp();
        if (lane == 0) mbar_wait(&sh.drain, 0, &never, status, 100000000ull);
        __syncwarp();
      }
    }
    else if (warp == 11 && busy) {
      // ------------------------------------------------------------ copies
      const bool split = p.log_bs == 7;  // a page has both halves
      const uint32_t bytes = split ? 64 * D : D << p.log_bs, per_half = split ? 1 : ppt / 2;
      const uint32_t to = smem_u32(smem) + C::kOffRaw + lane * bytes;
      uint32_t n = 0;
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        const Segment g = segment(k);
        const uint32_t end = n + 2 * (g.j1 - g.j0);
#pragma unroll 1
        for (; n < end; ++n) {
          const int ms = (n >> 1) % kMetaStages, st = n % kHalfStages, h = n & 1;
          if (h == 0) ok = wait_bar(&sh.meta_full[ms], ((n >> 1) / kMetaStages) & 1);
          if (ok && n >= (uint32_t)kHalfStages) ok = wait_bar(&sh.kv_empty[st], ((n / kHalfStages) - 1) & 1);
          if (!ok) break;
          const uint32_t valid = split ? sh.valid[ms] : sh.valid[ms] >> (h * per_half) & ((1u << per_half) - 1u);
          if (lane == 0) mbar_arrive_expect_tx(&sh.raw_full[st], __popc(valid) * bytes);
          __syncwarp();
          if ((valid >> lane) & 1)
            bulk_load(to + (st >> 1) * C::kRawStride + h * 64 * D, split ? sh.meta[ms][0].rows + h * 64 * D : sh.meta[ms][h * per_half + lane].rows,
                      bytes, &sh.raw_full[st]);
          __syncwarp();
        }
        if (g.last()) break;
      }
      // copies in flight end in any case; none may outlive the CTA
      volatile int never = 0;
#pragma unroll 1
      for (uint32_t t = n > (uint32_t)kHalfStages ? n - kHalfStages : 0; t < n; ++t)
        if (lane == 0) mbar_wait(&sh.raw_full[t % kHalfStages], (t / kHalfStages) & 1, &never, status, 100000000ull);
      __syncwarp();
    }
  } else if (warp >= 4) {
    setmaxnreg_dec<C::kRegsConv>();
    if (busy) {
      // ------------------------------------------------------------ converter
      // A thread takes 16-byte pieces (16 values) of rows kRowStep apart.  Of 8
      // neighbouring lanes 4 have pieces of one row and 4 of the next, with
      // columns 0 .. 63 of the one and 64 .. 127 of the other, so that what they
      // load and what they store falls into different banks.
      constexpr int kRowStep = kWG * 16 / D, kPer = 64 / kRowStep;  // of a half
      const int ct = tid - kWG;
      const int ch = D == 128 ? (ct & 3) | (((ct >> 2) ^ (ct >> 3)) & 1) << 2 : ct & 3;
      const int row0 = D == 128 ? ((ct >> 2) & 1) | ((ct >> 3) & ~1) : ct >> 2;
      const uint32_t row_lanes = D == 128 ? 0x0f0fu << (lane & 20) : 0xfu << (lane & 28);  // of the thread's row
      const uint32_t from0 = smem_u32(smem) + C::kOffRaw + row0 * D + ch * 16;
      const uint32_t to0 = smem_u32(smem) + (ch >> 2) * kHalfTile + row0 * 128;
      const uint32_t swz0 = (((2 * (ch & 3)) ^ (row0 & 7)) << 4);  // the other piece's differs in one bit
      static_assert(kRowStep % 8 == 0, "a thread's rows have one swizzle");
      const int q_row = ct % NQ, copy = ct / NQ;
      // q of a group into shared memory: D / 8 neighbouring lanes copy a row's
      // 16-byte pieces as they are, asynchronously; rows beyond the group's are
      // zero.
      constexpr int kLanes = D / 8, step = kWG / kLanes;  // rows at a time
      const int q_ch = ct % kLanes, c0q = ct / kLanes;
      const uint32_t dst = smem_u32(smem) + C::kOffQ + (q_ch >> 3) * kHalfTile;
      auto copy_q = [&](const Segment &g) {
        const int nq = real_columns(p, g.npos, g.slice());
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + ((size_t)g.row0 * p.H + g.slice() * p.HS) * D + q_ch * 8;
#pragma unroll 1
        for (int c = c0q; c < NQ; c += step)
          cp_async_16(dst + c * 128 + (((q_ch & 7) ^ (c & 7)) << 4), c < nq ? q + (size_t)c * D : q, c < nq ? 16 : 0);
      };
      copy_q(segment(0));
      uint32_t n = 0;
      // no way out when a wait has given up: the warps meet at barriers
#pragma unroll 1
      for (int k = 0;; ++k) {
        const Segment g = segment(k);
        const uint32_t end = n + 2 * (g.j1 - g.j0);
        // q of the first group comes before its keys do; that of a later one has to
        // wait for the last group's scores, its first tile has not
        const uint32_t q_at = k == 0 ? 0 : n + 2;
#pragma unroll 1
        for (;; ++n) {
          if (n == q_at) {
            // bf16 -> fp16 with a factor for each row, by the row's thread (its
            // copies share the work): the largest |q| becomes 224 .. 448; a
            // negative scale goes into q's sign (of a row with an infinity nothing
            // but NaN comes, whatever the factor)
            if (k > 0) {
              // the last group's scores have been made and its factors read
              (void)wait_bar(&sh.q_read, (k - 1) & 1);
              (void)wait_bar(&sh.s_full[1], ((q_at >> 1) - 2) & 1);
              copy_q(g);
            }
            cp_async_wait();
            named_bar_sync(kBarQ, kWG);
            const uint32_t q_at_row = smem_u32(smem) + C::kOffQ + q_row * 128;
            auto piece_at = [&](int c) { return q_at_row + (c >> 3) * kHalfTile + (((c & 7) ^ (q_row & 7)) << 4); };
            uint32_t amax = 0;
#pragma unroll 4
            for (int c = 0; c < kLanes; ++c) {
              uint32_t w[4];
              ld_shared(piece_at(c), w);
              amax = bf16x2_max(amax, bf16x2_max(bf16x2_max(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                                 bf16x2_max(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu)));
            }
            const int ex = scale_exponent(__uint_as_float(max(amax & 0xffffu, amax >> 16) << 16), kLeastQExp);
            const float inv = p.scale < 0.f ? -exp2_int(-ex) : p.scale > 0.f ? exp2_int(-ex) : 0.f;
            if (copy == 0) sh.q_factor[q_row] = exp2_int(ex) * fabsf(p.scale) * 1.4426950408889634f;
            if constexpr (C::kCopies > 1) named_bar_sync(kBarQ, kWG);
            const uint64_t inv2 = f32x2(__float_as_uint(inv), __float_as_uint(inv));
            constexpr int kOwn = kLanes / C::kCopies;  // pieces of each copy
#pragma unroll(kOwn < 2 ? kOwn : 2)
            for (int i = 0; i < kOwn; ++i) {
              const uint32_t at = piece_at(copy * kOwn + i);
              uint32_t w[4], f[4];
              ld_shared(at, w);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float lo, hi;
                f32x2_split(fmul2(f32x2(w[e] << 16, w[e] & 0xffff0000u), inv2), lo, hi);
                f[e] = f16x2_rn(lo, hi);
              }
#pragma unroll
              for (int y = 0; y < C::kCopies; ++y) st_shared(at + y * NQ * 128, f[0], f[1], f[2], f[3]);
            }
            fence_async_smem();
            mbar_arrive(&sh.q_full);
          }
          if (n == end) break;
          const int ms = (n >> 1) % kMetaStages, st = n % kHalfStages, h = n & 1;
          (void)wait_bar(&sh.raw_full[st], (n / kHalfStages) & 1);
          const uint32_t valid = sh.valid[ms];
          const bool look = !((sh.all_seen[ms] >> h) & 1), full = valid == (1u << ppt) - 1u;
          const uint32_t from = from0 + (st >> 1) * C::kRawStride + h * 64 * D, to = to0 + (st >> 1) * C::kStageBytes + h * 8192;
          uint32_t raw[kPer][4];
#pragma unroll
          for (int i = 0; i < kPer; ++i) ld_shared(from + i * kRowStep * D, raw[i]);
          if (!full) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              const int row = h * 64 + row0 + i * kRowStep;
              if (!((valid >> (row >> p.log_bs)) & 1)) raw[i][0] = raw[i][1] = raw[i][2] = raw[i][3] = 0;
            }
          }
          if (look) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              const uint32_t nan = __ballot_sync(0xffffffffu, nan_bytes(make_uint4(raw[i][0], raw[i][1], raw[i][2], raw[i][3])) != 0);
              if (nan & row_lanes) {
                // NaN in a row that not every row of the group sees
                const int row = h * 64 + row0 + i * kRowStep;
                if (sh.meta[ms][row >> p.log_bs].kind != kAllSeen) {
                  raw[i][0] = raw[i][1] = raw[i][2] = raw[i][3] = 0;
                  if (ch == 0) {
                    atomicOr(&sh.nan_keys[ms][row >> 5], 1u << (row & 31));
                    sh.nan_any[ms] = 1;
                  }
                }
              }
            }
          }
          __syncwarp();  // rows of 128 bytes are overwritten; all their pieces are a warp's
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            uint32_t f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_f16(raw[i][e], f[2 * e], f[2 * e + 1]);
            const uint32_t factor = sh.meta[ms][(h * 64 + row0 + i * kRowStep) >> p.log_bs].factor;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f16x2_mul(f[e], factor);
            const uint32_t at = to + i * kRowStep * 128;
            st_shared(at + swz0, f[0], f[1], f[2], f[3]);
            st_shared(at + (swz0 ^ 16), f[4], f[5], f[6], f[7]);
          }
          fence_async_smem();
          mbar_arrive(&sh.kv_full[st]);
        }
        if (g.last()) break;
      }
    }
  } else {
    setmaxnreg_inc<C::kRegsSoft>();
    if (ntiles < 0) {
      // the schedule was refused
      const size_t rows = (size_t)p.N * p.H;
      const uint4 nan4 = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
#pragma unroll 1
      for (size_t i = (size_t)blockIdx.x * kWG + tid; i < rows * (D / 8); i += (size_t)gridDim.x * kWG)
        reinterpret_cast<uint4 *>(p.out)[i] = nan4;
#pragma unroll 1
      for (size_t i = (size_t)blockIdx.x * kWG + tid; i < rows; i += (size_t)gridDim.x * kWG)
        p.lse[i] = __int_as_float(0x7fc00000);
    } else if (busy) {
      // ------------------------------------------------------------ softmax
      // Rows beyond the group's are zero in Q: their results are not written.
      constexpr int kSpan = C::kSpan;
      const int row = tid % NQ, copy = tid / NQ;  // row of the group
      const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
      uint32_t n = 0;
#pragma unroll 1
      for (int k = 0;; ++k) {
        const Segment g = segment(k);
        const int nreal = real_columns(p, g.npos, g.slice());
        const int pos = g.pos0 + (row < nreal ? row / p.HS : 0);
        // what the row sees: raw keys [raw_lo, pos], entries [0, entries)
        const int raw_lo = pos - p.W + 1, entries = (pos + 1) / p.m;
        float m_run = -INFINITY, m_use = 0.f, l_run = 0.f;  // m_use: what is subtracted
        int unit = 0;                                       // exponent of O
        (void)wait_bar(&sh.q_full, k & 1);
        const float cs = sh.q_factor[row];
        mbar_arrive(&sh.q_read);
#pragma unroll 1
        for (int j = g.j0; j < g.j1; ++j, ++n) {
          const int ms = n % kMetaStages;
          const PageMeta *meta = sh.meta[ms];
          (void)wait_bar(&sh.meta_full[ms], (n / kMetaStages) & 1);
          const int all_seen = sh.all_seen[ms], odd = sh.odd[ms];
          // positive and finite: a masked score stays -inf, that of a row of zeros 0
          const float ck = fminf(fmaxf(cs * exp2_int(sh.unit[ms]), FLT_MIN), FLT_MAX);
          if (odd >> 1) {
            // O in the tile's unit, once it holds the last tile's keys
            (void)wait_bar(&sh.pv_done[1], (n - 1) & 1);
            tc_fence_after();
            scale_o<D>(lane_addr + kColO, exp2_int(odd >> 1));
          }
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            (void)wait_bar(&sh.s_full[h], n & 1);
            tc_fence_after();
            const int k0 = h * 64 + copy * kSpan;  // first of the thread's keys, uniform in a warp
            if (odd & 1) scale_s<kSpan>(lane_addr + k0, meta, k0, p.log_bs);
            uint32_t sv[kSpan];
            if constexpr (kSpan == 16) {
              tmem_ld16(lane_addr + k0, sv);
            } else {
#pragma unroll
              for (int c = 0; c < kSpan; c += 32) tmem_ld32(lane_addr + k0 + c, *reinterpret_cast<uint32_t(*)[32]>(sv + c));
            }
            // which of them the row sees
            const bool plain = (all_seen >> h) & 1;
            if (!plain) (void)wait_bar(&sh.kv_full[(2 * n + h) % kHalfStages], (n / kStages) & 1);  // for the converter's notes
            const bool odd_rows = sh.nan_any[ms] != 0;
            uint64_t vis = ~0ull;
            if (!plain) {
              vis = 0;
              const int bs = 1 << p.log_bs;
#pragma unroll 1
              for (int at = 0; at < kSpan; at += bs) {
                const PageMeta &pm = meta[(k0 + at) >> p.log_bs];
                const int skip = (k0 + at) & (bs - 1), cnt = min(bs, kSpan);
                const int kind = pm.kind, key = pm.key0 + skip;  // key of column `at`
                // of columns [at, at + cnt): those with a visible key
                int a = 0, b = kind == kAllSeen ? cnt : 0;
                if (kind == kRaw) {
                  a = max(raw_lo - key, 0);
                  b = min(pos - key + 1, cnt);
                } else if (kind == kComp) {
                  b = min(entries - key, cnt);
                }
                if (b > a) vis |= (b - a >= 64 ? ~0ull : ((1ull << (b - a)) - 1ull)) << (at + a);
              }
            }
            if (odd_rows) {
              uint64_t bad = sh.nan_keys[ms][k0 >> 5] >> (k0 & 31);
              if (kSpan == 64) bad |= (uint64_t)sh.nan_keys[ms][(k0 >> 5) + 1] << 32;
              if constexpr (kSpan < 64) bad &= (1ull << kSpan) - 1;
              if (bad & vis) l_run = __int_as_float(0x7fc00000);
            }
            tmem_wait_ld();
            if (!plain) {
              constexpr int kStep = kSpan < 32 ? kSpan : 32;
              constexpr uint32_t kAll = kStep == 32 ? 0xffffffffu : (1u << kStep) - 1u;
#pragma unroll
              for (int c = 0; c < kSpan; c += kStep) {
                const uint32_t v = (uint32_t)(vis >> c) & kAll;
                if (!__all_sync(0xffffffffu, v == kAll)) {
#pragma unroll
                  for (int y = 0; y < kStep; ++y)
                    if (!((v >> y) & 1)) sv[c + y] = 0xff800000u;
                }
              }
            }
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int y = 0; y < kSpan; y += 4) {
              m0 = fmax3(m0, __uint_as_float(sv[y]), __uint_as_float(sv[y + 1]));
              m1 = fmax3(m1, __uint_as_float(sv[y + 2]), __uint_as_float(sv[y + 3]));
            }
            const float mx = fmaxf(m0, m1) * ck;
            // raise the reference (seldom); the sums made with the old one follow
            const bool raise = mx > m_run + kRaiseLog2;  // at first: any key that is seen
            if (__any_sync(0xffffffffu, raise)) {
              const bool had = raise && m_run > -INFINITY;  // else O holds nothing of this row yet
              const float f = had ? ex2_approx(m_run - mx) : 1.f;
              l_run *= f;
              if (raise) m_run = mx;
              m_use = m_run == -INFINITY ? 0.f : m_run - kBias;
              if (__any_sync(0xffffffffu, had)) {
                // O holds the sum up to the keys before these once that is done
                (void)wait_bar(&sh.pv_done[h ^ 1], (h ? n : n - 1) & 1);
                tc_fence_after();
                constexpr int kPart = kSpan == 64 ? 16 : 32;  // columns that fit the registers beside the scores
#pragma unroll 1
                for (int c = 0; c < D; c += kPart) {
                  uint32_t o[kPart];
                  if constexpr (kPart == 16) tmem_ld16(lane_addr + kColO + c, o);
                  else tmem_ld32(lane_addr + kColO + c, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int y = 0; y < kPart; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                  if constexpr (kPart == 16) tmem_st16(lane_addr + kColO + c, o);
                  else tmem_st32(lane_addr + kColO + c, o);
                }
              }
            }
            // P over the first columns of the half's S, with zeros for the other
            // copies' keys
            const uint32_t pcol = lane_addr + h * 64;
            if (odd & 1) {
              // the masked scores go back to tensor memory
              if constexpr (kSpan == 16) {
                tmem_st16(lane_addr + k0, sv);
              } else {
#pragma unroll
                for (int c = 0; c < kSpan; c += 32) tmem_st32(lane_addr + k0 + c, *reinterpret_cast<uint32_t(*)[32]>(sv + c));
              }
              tmem_wait_st();
              l_run += scaled_p<kSpan>(lane_addr + k0, pcol + copy * (kSpan / 2), ck, m_use, meta, k0, p.log_bs);
            } else {
              uint32_t pk[kSpan / 2];
              const uint64_t ck2 = f32x2(__float_as_uint(ck), __float_as_uint(ck));
              const uint64_t nm2 = f32x2(__float_as_uint(-m_use), __float_as_uint(-m_use));
              uint64_t acc[2] = {0, 0};
#pragma unroll
              for (int c4 = 0; c4 < kSpan / 16; ++c4) {
#pragma unroll
                for (int y = 0; y < 16; y += 2) {
                  float t0, t1;
                  f32x2_split(ffma2(f32x2(sv[c4 * 16 + y], sv[c4 * 16 + y + 1]), ck2, nm2), t0, t1);
                  const float e0 = ex2_approx(t0), e1 = ex2_approx(t1);
                  acc[(y >> 1) & 1] = fadd2(acc[(y >> 1) & 1], f32x2(__float_as_uint(e0), __float_as_uint(e1)));
                  pk[c4 * 8 + (y >> 1)] = f16x2_rn(e0, e1);
                }
                if (kSpan > 16 && (c4 & 1)) tmem_st16(pcol + copy * (kSpan / 2) + (c4 - 1) * 8, *reinterpret_cast<uint32_t(*)[16]>(&pk[(c4 - 1) * 8]));
              }
              if constexpr (kSpan == 16) tmem_st8(pcol + copy * 8, pk);
              float a, b;
              f32x2_split(fadd2(acc[0], acc[1]), a, b);
              l_run += a + b;
            }
            if constexpr (C::kCopies == 2) {
              uint32_t zero[16];
#pragma unroll
              for (int y = 0; y < 16; ++y) zero[y] = 0;
              tmem_st16(pcol + (copy ^ 1) * 16, zero);
            }
            if constexpr (C::kCopies == 4) {
              uint32_t zero[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) zero[y] = 0;
#pragma unroll
              for (int y = 1; y < 4; ++y) tmem_st8(pcol + ((copy + y) & 3) * 8, zero);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.p_full[h]);
          }
          unit = sh.unit[ms];
          mbar_arrive(&sh.meta_empty[ms]);
        }
        m_run -= kBias;  // what the sums are relative to
        if (*abort_flag) l_run = __int_as_float(0x7fc00000);
        const bool whole = g.slot < 0;
        const size_t orow = (size_t)g.row0 * p.H + g.slice() * p.HS;  // rows of the group are rows of q and out in order
        float weight = 1.f;
        if constexpr (C::kCopies > 1) {
          // the copies' common reference and sum
          sh.ml[tid] = make_float2(m_run, l_run);
          named_bar_sync(kBarOut, kWG);
          float M = -INFINITY, L = 0.f;
#pragma unroll
          for (int y = 0; y < C::kCopies; ++y) M = fmaxf(M, sh.ml[row + y * NQ].x);
#pragma unroll
          for (int y = 0; y < C::kCopies; ++y) {
            const float2 v = sh.ml[row + y * NQ];
            const float f = v.x == -INFINITY ? 0.f : ex2_approx(v.x - M);
            L += v.y != 0.f ? f * v.y : 0.f;  // NaN stays
            if (y == copy) weight = f;
          }
          if (l_run != l_run) L = l_run;
          m_run = M;
          l_run = L;
        }
        if (row < nreal && copy == 0) {
          if (whole) p.lse[orow + row] = (m_run + log2f(l_run)) * 0.69314718055994531f;
          else p.part_ml[(size_t)g.slot * NQ + row] = make_float2(m_run, l_run);
        }
        if (!whole && tid == 0) p.part_unit[g.slot] = unit;
        const float inv = weight * (whole ? exp2_int(unit) / l_run : 1.f);
        (void)wait_bar(&sh.pv_done[1], (n - 1) & 1);
        tc_fence_after();
        // O leaves through shared memory, 64 bytes of a row at a time, so that
        // four lanes write a row's: a store to 32 rows takes 32 cycles.
        uint8_t *to = whole ? static_cast<uint8_t *>(p.out) + orow * D * 2 : reinterpret_cast<uint8_t *>(p.part_o + (size_t)g.slot * NQ * D);
        const int row_bytes = whole ? D * 2 : D * 4, piece = lane & 3;
        const uint32_t join = smem_u32(sh.join);
        const uint32_t mine = join + tid * 64, swz = (tid >> 1) & 3;
        const bool packed = C::kCopies == 1 && whole;  // staged as bf16 already: 32 columns
        const int rounds = packed ? D / 32 : D / 16;
#pragma unroll 1
        for (int c = 0; c < rounds; ++c) {
          uint32_t o[16];
          if (packed) {
            uint32_t x[32];
            tmem_ld32(lane_addr + kColO + c * 32, x);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = pack_bf16x2(__uint_as_float(x[2 * y]) * inv, __uint_as_float(x[2 * y + 1]) * inv);
          } else {
            tmem_ld16(lane_addr + kColO + c * 16, o);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * inv);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) st_shared(mine + ((y ^ swz) << 4), o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          if constexpr (C::kCopies == 1) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = warp * 32 + i * 8 + (lane >> 2);
              uint32_t v[4];
              ld_shared(join + r * 64 + ((piece ^ ((r >> 1) & 3)) << 4), v);
              if (r < nreal) *reinterpret_cast<uint4 *>(to + (size_t)r * row_bytes + c * 64 + piece * 16) = make_uint4(v[0], v[1], v[2], v[3]);
            }
            __syncwarp();
          } else {
            named_bar_sync(kBarOut, kWG);
#pragma unroll
            for (int i = 0; i < NQ / 32; ++i) {
              const int r = i * 32 + (tid >> 2);
              float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int x = 0; x < C::kCopies; ++x) {
                uint32_t v[4];
                ld_shared(join + (r + x * NQ) * 64 + ((piece ^ ((r >> 1) & 3)) << 4), v);
#pragma unroll
                for (int y = 0; y < 4; ++y) sum[y] += __uint_as_float(v[y]);
              }
              uint8_t *at = to + (size_t)r * row_bytes;
              if (r < nreal) {
                if (whole) *reinterpret_cast<uint2 *>(at + c * 32 + piece * 8) = make_uint2(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]));
                else *reinterpret_cast<float4 *>(at + c * 64 + piece * 16) = make_float4(sum[0], sum[1], sum[2], sum[3]);
              }
            }
            named_bar_sync(kBarOut, kWG);
          }
        }
        tc_fence_before();
        if (g.last()) break;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sh.abort) atomicExch(status, HCA_ERR_TIMEOUT);
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

template <int NQ, int D>
cudaError_t launch(const AttnParams &p, cudaStream_t st) {
  using C = Cfg<NQ, D>;
  static SmemAttrOnce attr;
  const cudaError_t e = attr.ensure(reinterpret_cast<const void *>(hca_cache_attn_kernel<NQ, D>), C::kSmem);
  if (e != cudaSuccess) return e;
  ProfScope prof(kKCacheAttn, st);
  if (!p.in_cta) return launch_behind(hca_cache_attn_kernel<NQ, D>, dim3(p.grid), kThreads, C::kSmem, st, p);
  hca_cache_attn_kernel<NQ, D><<<p.grid, kThreads, C::kSmem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

namespace cache {

int tc_cache_ctas() { return 2; }
int tc_cache_threads() { return kThreads; }

cudaError_t tc_cache_attn(const AttnParams &p, cudaStream_t st) {
  const int which = (p.NQ == 32 ? 0 : p.NQ == 64 ? 1 : 2) + (p.D == 64 ? 3 : 0);
  switch (which) {
    case 0: return launch<32, 128>(p, st);
    case 1: return launch<64, 128>(p, st);
    case 2: return launch<128, 128>(p, st);
    case 3: return launch<32, 64>(p, st);
    case 4: return launch<64, 64>(p, st);
    default: return launch<128, 64>(p, st);
  }
}

}  // namespace cache
}  // namespace hca
