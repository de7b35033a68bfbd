// hca_cache_shared.cu -- attention over the 8-bit cache for requests that begin
// with the same compressed entries: the common ones once for all of them.
//
// The rows of q of a prefix's requests are adjacent, and every one of them sees
// every common entry, so that part is dense attention of one matrix of rows over
// one list of pages, without masks:
//   S [256 x 128 keys] = Q K^T,  O [256 x D] += P K     kind::f16 (tcgen05)
// A request by itself fills 64 of the tensor cores' 128 rows with a token of 64
// heads, and each request converts the entries to fp16 for itself.  Here tiles
// are full, and an entry is converted once for 256 rows.
//
// The work.  A prefix of `rows` rows and `tiles` key tiles is ceil(rows / 256) row
// tiles of `tiles` units; all units of all prefixes form one line, cut into equal
// ranges, one for each CTA.  What a CTA has of a row tile (a segment) leaves a
// partial result: O / l in fp32, the reference exponent and the sum l.  The
// requests' own keys (window and entries behind the prefix) go through the kernels
// of hca_cache_attn, which leave fp32 rows, and the join kernel adds up.
//
// A CTA has two tiles A and B of 128 rows and one stream of keys, 512 threads:
//   warps 0 - 3, 4 - 7   softmax of A, of B: a thread has a row
//   warps 8 - 11         converter: e4m3 -> fp16 key tiles
//   warp 12              pages: block ids and scales, looked up ahead
//   warps 13, 14         MMA issuers of A and of B
//   warp 15              tensor memory
// S of a tile is 128 columns of tensor memory, softmaxed in two halves of 64 keys
// whose P (fp16) takes the first half of their columns: the first half's product
// with K runs while the second half is worked on, and one tile's products while
// the other tile's softmax runs.  Numbers are as in hca_cache_attn_tc.cu: q as
// fp16 with a power of two for each row, keys as k8 * 2^e in units of 2^u, u the
// largest scale of the segment's pages; what is left of a scale (below 2^-15 of
// the unit, or no power of two) multiplies scores and probabilities.
//
// Bounds.  164,544 rows (2,571 tokens of 64 heads) over 9,984 entries, 841 GFLOP: 518 us,
// 1.62 PFLOP/s, 83% of the measured rate of a plain product; tensor pipe 70% active, 2.07
// instructions a cycle.  A step of 256 rows x 128 keys takes 1.57 us: 64-key scores are
// bound by shared memory (48 cycles a product where the pipe needs 32), and a half's
// score -> softmax -> output has three hand-overs.  Beside it the requests' own keys 118 us
// and the join 25: 657 us in all, 764 without sharing.  4,096 rows over 24,960 entries, 16
// row tiles in 128 ranges: 58 us, 94 without sharing (calls in a graph, as all figures here
// and below; between boxes they differ by 2%); 40 are steps, 8 the beginning (table,
// scales, first keys), 3 the way out, 7 the join.
//   Slower (each against the kernel of its time): S of 128 keys at once 646 to 686 us, 585
// in halves; q in tensor memory 768 for 646; pages by bulk copies and converted from
// shared memory 585 for 567; products issued by warps that wait together 562 for 555; the
// maximum inside the exponentials' loop 591 for 583; all row tiles through the join 86 us
// of join for 33.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <climits>

#include "hca_cache_attn.cuh"
#include "hca_cache_tc.cuh"

namespace hca {
using namespace tc;
using namespace cache;

namespace {

constexpr int kSharedMaxGroups = 256, kMaxGrid = 256, kPadded = 6;
constexpr int kWG = 128, kThreads = 4 * kWG;
constexpr int kMetaStages = 8, kKvStages = 4;
constexpr int kRegsSoft = 168, kRegsConv = 88, kRegsIssue = 88;
static_assert(2 * kRegsSoft + kRegsConv + kRegsIssue <= 4 * 128, "register split must fit the launch");
constexpr uint32_t kTmem = 512;
// S of tile x and half h (P takes the first half of its columns), O of tile x
__device__ __forceinline__ constexpr uint32_t col_s(int x, int h) { return 128u * x + 64u * h; }
__device__ __forceinline__ constexpr uint32_t col_o(int x) { return 256u + 128u * x; }

struct Table;

struct SharedParams {
  SharedAttnParams own;  // of the requests' own keys
  Table *table;          // what the prefixes' kernel went by
  int32_t *err;          // [grid]
  float2 *part_ml;       // [slots][256] reference exponent and sum
  float *part_o;         // [slots][256][D]
  const float *own_out, *own_lse;
  int32_t *status;
  __nv_bfloat16 *out;
  float *lse;
  int grid;              // CTAs of the prefixes' kernel
  int stall;
  int merge;             // the requests' own keys are done: row tiles that are not cut are finished here
};

// A prefix with its rows and its place in the line.
struct Prefix {
  int row0, rows;   // rows of q and out
  int tiles, pages; // key tiles, pages
  int span;         // units that a row tile takes of the line: its key tiles, or more (below)
  int line0, rt0;   // first unit, first row tile
  int request;      // whose compressed table is read
};

struct Table {
  int units;            // of the line, -1: the prefixes are refused
  int quota;            // units of a CTA
  int row_tiles;        // of all prefixes, those without common entries among them
  Prefix g[kSharedMaxGroups];
};

// The line, by all threads of a block.  `tmp` holds a value for each warp.
//
// A CTA that has the end of one row tile and the beginning of the next pays for an
// epilogue, a q and a pipeline that fills again, about kPadded - 1 units' time.  So
// where row tiles can be cut into pieces of up to that much more than an equal
// share, each CTA gets one piece (the line has gaps then: `span`).
__device__ __forceinline__ void make_table(const SharedParams &p, Table &t, long long *tmp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  bool ok = true;
  long long units = 0, nrt = 0;
  if (warp == 0) {
    for (int g = lane; g < p.own.G; g += 32) {
      PrefixSize z;
      const bool fine = prefix_size(p.own, g, z);
      ok = ok && fine;
      int r = 0;
      if (fine) {
        // the first that has tokens: the last one that begins where the prefix does
        r = p.own.first[g];
        const int s0 = p.own.start[r];
        for (int end = p.own.first[g + 1]; end - r > 1;) {
          const int mid = (r + end) >> 1;
          if (p.own.start[mid] <= s0) r = mid; else end = mid;
        }
      }
      t.g[g] = Prefix{z.row0, z.rows, z.tiles, fine ? p.own.cols[g] : 0, z.tiles, 0, 0, r};
      units += (long long)z.row_tiles() * z.tiles;
      nrt += z.row_tiles();
    }
    units = warp_sum(units);
    nrt = warp_sum(nrt);
    ok = __all_sync(0xffffffffu, ok) && units < kMaxTiles;
  } else if (p.own.beside) {
    const long long own = warp_sum(own_tiles(p.own, tid - 32, blockDim.x - 32));
    if (lane == 0) tmp[warp] = own;
  }
  __syncthreads();
  if (warp == 0) {
    int ctas = p.grid;
    if (p.own.beside) {
      const long long own = warp_sum(lane > 0 && lane < warps ? tmp[lane] : 0);
      ctas = max(prefix_sms(p.own, ok ? units : 0, own), 1);
    }
    int quota = max((int)(((ok ? units : 0) + ctas - 1) / ctas), 1);
    if (ok) {
      // a part more costs the join about an eighth of a unit
      int longest = 0;
      for (int g = lane; g < p.own.G; g += 32) longest = max(longest, t.g[g].tiles);
      longest = __reduce_max_sync(0xffffffffu, longest);
      quota = max(quota, (int)sqrtf((float)longest * (1.f / 8.f)));
    }
    bool pad = false;
    if (ok && nrt <= ctas) {  // else there are more row tiles than CTAs
      int pieces[kPadded] = {};
      for (int g = lane; g < p.own.G; g += 32) {
        const int n = (t.g[g].rows + kRowTile - 1) / kRowTile;  // at most kMaxGrid
#pragma unroll
        for (int k = 0; k < kPadded; ++k) pieces[k] += n * min((t.g[g].tiles + quota + k - 1) / (quota + k), kMaxGrid + 1);
      }
#pragma unroll
      for (int k = kPadded - 1; k >= 0; --k) pieces[k] = __reduce_add_sync(0xffffffffu, pieces[k]);
      int more = kPadded;  // the least that fits
#pragma unroll
      for (int k = kPadded - 1; k >= 0; --k)
        if (pieces[k] <= ctas) more = k;
      pad = more < kPadded;
      if (pad) quota += more;
    }
    int line = 0, rt = 0;
    for (int g0 = 0; ok && g0 < p.own.G; g0 += 32) {
      const int g = g0 + lane;
      int n = 0, span = 0;
      if (g < p.own.G) {
        n = (t.g[g].rows + kRowTile - 1) / kRowTile;
        span = pad ? (t.g[g].tiles + quota - 1) / quota * quota : t.g[g].tiles;
      }
      int a = n, b = n * span;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) a += x, b += y;
      }
      if (g < p.own.G) {
        t.g[g].span = span;
        t.g[g].rt0 = rt + a - n;
        t.g[g].line0 = line + b - n * span;
      }
      rt += __shfl_sync(0xffffffffu, a, 31);
      line += __shfl_sync(0xffffffffu, b, 31);
    }
    if (lane == 0) {
      t.units = ok ? line : -1;
      t.quota = quota;
      t.row_tiles = rt;
    }
    __syncwarp();
    if (blockIdx.x == 0) {  // for the join
      if (lane == 0) {
        p.table->units = t.units;
        p.table->quota = quota;
        p.table->row_tiles = rt;
      }
      for (int g = lane; g < p.own.G; g += 32) p.table->g[g] = t.g[g];
    }
  }
  __syncthreads();
}

// What a CTA has of a row tile.
struct Part {
  int row0, rows;      // rows of q
  int j0, j1;          // key tiles
  int slot;
  int pages, request;
  bool whole;          // all key tiles of the row tile
  bool last;           // of the CTA's
};

struct Walk {
  int u, end, g;
  __device__ __forceinline__ Part next(const Table &t, int cta) {
    while (u >= t.g[g].line0 + (t.g[g].rows + kRowTile - 1) / kRowTile * t.g[g].span) ++g;
    const Prefix &x = t.g[g];
    const int rt = (u - x.line0) / x.span;
    Part s;
    s.j0 = u - x.line0 - rt * x.span;
    const int n = min(x.span - s.j0, end - u);
    s.j1 = min(x.tiles, s.j0 + n);
    s.whole = s.j0 == 0 && s.j1 == x.tiles;
    s.row0 = x.row0 + rt * kRowTile;
    s.rows = min(kRowTile, x.rows - rt * kRowTile);
    s.slot = x.rt0 + rt + cta;
    s.pages = x.pages;
    s.request = x.request;
    u += n;
    s.last = u >= end;
    return s;
  }
};

__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ void prefetch_line(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory"); }

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kStageBytes = kHalves * kHalfTile;  // fp16 tile of 128 keys, or of 128 rows of q
  static constexpr int kOffQ = kKvStages * kStageBytes;
  static constexpr int kSmem = kOffQ + 2 * kStageBytes + 1024;
};

struct TileMeta {
  const uint8_t *rows[8];  // NULL: no page, or a bad one
  uint32_t factor[8];      // 2^e of its keys, for both values of a pair of fp16
  float rest[8];           // the page's scale is 2^(unit + e) * rest
  uint32_t valid;          // pages that are there
  int keys;                // keys of the tile
  int unit;
  int odd, bad;            // some rest is not 1; a bad block id or scale
};

struct Shared {
  uint4 out[2 * kWG * 4];  // O on its way out: 64 bytes of each row
  float own[kRowTile];     // what a row's own part counts
  uint64_t meta_full[kMetaStages], meta_empty[kMetaStages];
  uint64_t kv_full[kKvStages], kv_empty[kKvStages];
  uint64_t q_full[2], s_full[2][2], p_full[2][2], pv_done[2][2], drain[2], never;
  TileMeta meta[kMetaStages];
  Table table;
  long long tmp[kThreads / 32];
  uint32_t tmem_base;
  int abort;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) hca_cache_prefix_kernel(const SharedParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  volatile int *abort_flag = &sh.abort;
  int32_t *status = &p.err[blockIdx.x];

  // what the schedule looks at, and this CTA's share of q, on their way to L2
  for (int r = tid * 32; r < p.own.R; r += kThreads * 32) {
    prefetch_line(p.own.start + r);
    prefetch_line(p.own.held + r);
  }
  if (tid == kThreads - 1) {
    prefetch_line(p.own.first);
    prefetch_line(p.own.cols);
    const size_t bytes = (size_t)p.own.N * p.own.H * D * 2, share = (bytes / gridDim.x + 15) & ~(size_t)15, at = share * blockIdx.x;
    if (!p.merge && at < bytes) prefetch_l2(static_cast<const uint8_t *>(p.own.q) + at, (uint32_t)min(share, bytes - at));
  }
  if (tid == 0) {
    for (int s = 0; s < kMetaStages; ++s) {
      mbar_init(&sh.meta_full[s], 1);
      mbar_init(&sh.meta_empty[s], 8);  // the softmax warps are the last to read a tile's pages
    }
    for (int s = 0; s < kKvStages; ++s) {
      mbar_init(&sh.kv_full[s], 4);
      mbar_init(&sh.kv_empty[s], 2);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh.q_full[x], 4);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sh.s_full[x][h], 1);
        mbar_init(&sh.p_full[x][h], 4);
        mbar_init(&sh.pv_done[x][h], 1);
      }
      mbar_init(&sh.drain[x], 1);
    }
    mbar_init(&sh.never, 1);
    sh.abort = 0;
    p.err[blockIdx.x] = HCA_OK;
    fence_mbar_init();
  }
  if (warp == 15) {
    tmem_alloc(&sh.tmem_base, kTmem);
    tmem_relinquish();
  }
  make_table(p, sh.table, sh.tmp);
  // The requests' own keys, where they run beside this: when every CTA has its tensor
  // memory, which those need too.
  pdl_launch_dependents();
  const int units = sh.table.units, quota = sh.table.quota;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(sh.tmem_base);
  const long long c0 = (long long)quota * blockIdx.x;
  const bool busy = c0 < units;
  const Walk from = {(int)c0, (int)min(c0 + quota, (long long)max(units, 0)), 0};

  const uint32_t limit_ns = (uint32_t)p.own.wait_ns;
  auto wait_bar = [&](uint64_t *bar, uint32_t parity) {  // mostly there already
    return __all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity) || mbar_wait_idle(bar, parity, abort_flag, limit_ns));
  };
  const int ppt = kTileKeys >> p.own.log_bs;  // pages of a tile: 1 .. 8
  if (warp >= 12) {
    setmaxnreg_dec<kRegsIssue>();
    if (warp == 12 && busy) {
      // ------------------------------------------------------------ pages
      const int batch = 32 / ppt;  // tiles whose pages the warp's lanes look up at once
      const uint32_t page_bytes = D << p.own.log_bs;
      Walk walk = from;
      uint32_t n = 0;
      bool ok = true;
      auto page_scale = [&](const Part &s, int page, int &id) {
        id = p.own.comp.table[(size_t)s.request * p.own.comp.cols + page];
        const bool in = id >= 0 && id < p.own.comp.nblocks;
        if (!in) id = -1;
        return in ? p.own.comp.scale[id] : 0.f;
      };
#pragma unroll 1
      for (bool last = false; ok && !last;) {
        const Part s = walk.next(sh.table, blockIdx.x);
        last = s.last;
        // the unit: the largest scale of the segment's pages
        int unit = INT_MIN;
        const int v0 = s.j0 * ppt, v1 = min(s.j1 * ppt, s.pages);
        int id = -1;  // of the lane's page of the next tiles
        float scale = 0.f;
        if (v0 + lane < v1) scale = page_scale(s, v0 + lane, id);
#pragma unroll 4
        for (int v = v0 + lane; v < v1; v += 32) {
          int other;
          const float sc = v < v0 + 32 ? scale : page_scale(s, v, other);
          float part;
          if (sc > 0.f && sc < INFINITY) unit = max(unit, split_scale(sc, part));
        }
        unit = __reduce_max_sync(0xffffffffu, unit);
        unit = unit == INT_MIN ? 0 : min(max(unit, kLeastUnit), kMostUnit);
#pragma unroll 1
        for (int jb = s.j0; ok && jb < s.j1; jb += batch) {
          const int v = jb * ppt + lane;
          const uint8_t *rows = nullptr;
          uint32_t factor = f16x2_exp2(0);
          float rest = 1.f;
          bool bad = false;
          if (v < v1) {
            if (jb > s.j0) scale = page_scale(s, v, id);
            bad = !(scale > 0.f && scale < INFINITY);
            if (!bad) {
              rows = p.own.comp.pool + (size_t)id * page_bytes;
              float part;
              const int ex = split_scale(scale, part), e = min(max(ex - unit, kLeastExp), kMostExp);
              factor = f16x2_exp2(e);
              rest = part * exp2_int(max(ex - unit - e, -120));
            }
          }
          const int jn = min(batch, s.j1 - jb);
#pragma unroll 1
          for (int t = 0; t < jn; ++t, ++n) {
            const int ms = n % kMetaStages;
            if (n >= (uint32_t)kMetaStages) ok = wait_bar(&sh.meta_empty[ms], ((n / kMetaStages) - 1) & 1);
            if (!ok) break;
            TileMeta &to = sh.meta[ms];
            const bool here = lane / ppt == t;
            if (here) {
              if (rows) prefetch_l2(rows, page_bytes);
              to.rows[lane % ppt] = rows;
              to.factor[lane % ppt] = factor;
              to.rest[lane % ppt] = rest;
            }
            const uint32_t valid = __ballot_sync(0xffffffffu, here && rows) >> (t * ppt);
            const bool odd = __any_sync(0xffffffffu, here && rest != 1.f), wrong = __any_sync(0xffffffffu, here && bad);
            if (lane == 0) {
              to.valid = valid;
              to.keys = min(ppt, s.pages - (jb + t) * ppt) << p.own.log_bs;
              to.unit = unit;
              to.odd = odd;
              to.bad = wrong;
              if (wrong) *status = HCA_ERR_CACHE;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.meta_full[ms]);
          }
        }
      }
    } else if ((warp == 13 || warp == 14) && busy) {
      // ------------------------------------------------------------ MMA of tile x
      // Its products run in order: S of half u + 2 is issued right behind the
      // O product of half u, whose P it overwrites.
      const int x = warp - 13;
      const uint32_t kv0 = smem_u32(smem), q0 = smem_u32(smem + C::kOffQ) + x * C::kStageBytes;
      const uint64_t dk = smem_desc_sw128(kv0, 16, 1024);         // K view of stage 0
      const uint64_t dv = smem_desc_sw128(kv0, kHalfTile, 1024);  // V view of stage 0
      const uint64_t dq = smem_desc_sw128(q0, 16, 1024);
      const uint32_t id_s = idesc_f16_f32(128, 64, false, false), id_o = idesc_f16_f32(128, D, false, true);
      if (elect_one()) {
        // by one thread from its waits to its products: a warp that looks at barriers
        // together and elects a thread for each step takes longer than the products
        Walk walk = from;
        uint32_t n = 0, nseg = 0;  // tiles, segments
        bool ok = true, issued = false;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
          return mbar_try_wait(smem_u32(bar), parity) || mbar_wait_idle(bar, parity, abort_flag, limit_ns);
        };
        if (p.stall && x == 0) ok = mbar_wait(&sh.never, 0, abort_flag, status, p.own.wait_ns);  // injected: nothing arrives
#pragma unroll 1
        for (bool last = false; ok && !last; ++nseg) {
          const Part s = walk.next(sh.table, blockIdx.x);
          last = s.last;
          const int halves = 2 * (s.j1 - s.j0);
          ok = wait(&sh.q_full[x], nseg & 1);
#pragma unroll 1
          for (int u = 0; ok && u < halves + 2; u += 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (u >= 2) {
                const uint32_t t = n + (u >> 1) - 1, st = t % kKvStages;
                ok = ok && wait(&sh.p_full[x][h], t & 1);
                if (ok) {
                  tc_fence_after();
                  const uint64_t bv = dv + desc_bytes(st * C::kStageBytes + h * 8192);
                  const uint32_t more = u > 2 || h > 0;
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) mma_ts(tmem + col_o(x), tmem + col_s(x, h) + kk * 8, bv + mnmaj_step(kk), id_o, more || kk > 0);
                  mma_commit(&sh.pv_done[x][h]);
                  if (h == 1) mma_commit(&sh.kv_empty[st]);
                }
              }
              if (u < halves) {
                const uint32_t t = n + (u >> 1), st = t % kKvStages;
                if (h == 0) ok = ok && wait(&sh.kv_full[st], (t / kKvStages) & 1);
                if (ok) {
                  tc_fence_after();
                  const uint64_t b = dk + desc_bytes(st * C::kStageBytes + h * 8192);
#pragma unroll
                  for (int kk = 0; kk < D / 16; ++kk) mma_ss(tmem + col_s(x, h), dq + kmaj_step(kk), b + kmaj_step(kk), id_s, kk > 0);
                  mma_commit(&sh.s_full[x][h]);
                  issued = true;
                }
              }
            }
          }
          n += halves / 2;
        }
        if (!ok && issued) {
          volatile int never = 0;
          mma_commit(&sh.drain[x]);
          mbar_wait(&sh.drain[x], 0, &never, status, 100000000ull);
        }
      }
      __syncwarp();
    }
  } else if (warp >= 8) {
    setmaxnreg_dec<kRegsConv>();
    if (busy) {
      // ------------------------------------------------------------ converter
      // A thread takes 16-byte pieces (16 values) of rows kRowStep apart.  Of 8
      // neighbouring lanes 4 have pieces of one row and 4 of the next, with
      // columns 0 .. 63 of the one and 64 .. 127 of the other, so that what they
      // load and what they store falls into different banks.
      constexpr int kRowStep = kWG * 16 / D, kPer = kTileKeys / kRowStep;
      const int ct = tid - 2 * kWG;
      const int ch = D == 128 ? (ct & 3) | (((ct >> 2) ^ (ct >> 3)) & 1) << 2 : ct & 3;
      const int row0 = D == 128 ? ((ct >> 2) & 1) | ((ct >> 3) & ~1) : ct >> 2;
      const uint32_t to0 = smem_u32(smem) + (ch >> 2) * kHalfTile + row0 * 128;
      const uint32_t swz0 = (((2 * (ch & 3)) ^ (row0 & 7)) << 4);  // the other piece's differs in one bit
      static_assert(kRowStep % 8 == 0, "a thread's rows have one swizzle");
      uint32_t tiles = 0;
      Walk walk = from;
      for (bool last = false; !last;) {
        const Part s = walk.next(sh.table, blockIdx.x);
        last = s.last;
        tiles += s.j1 - s.j0;
      }
      // Piece i of a tile, from memory (zero where there is no page).  When a wait has
      // given up the tile's pages may never have been looked up: nothing is read then.
      bool ok = true;
      auto piece = [&](const TileMeta &meta, int i, uint4 &w) {
        const int row = row0 + i * kRowStep, page = row >> p.own.log_bs;
        const uint8_t *rows = ok ? meta.rows[page] : nullptr;
        w = make_uint4(0, 0, 0, 0);
        if (rows) w = *reinterpret_cast<const uint4 *>(rows + (row - (page << p.own.log_bs)) * D + ch * 16);
      };
      uint4 raw[kPer];
      ok = wait_bar(&sh.meta_full[0], 0);
#pragma unroll
      for (int i = 0; i < kPer; ++i) piece(sh.meta[0], i, raw[i]);
      // no way out when a wait has given up: the softmax goes on too
#pragma unroll 1
      for (uint32_t n = 0; n < tiles; ++n) {
        const TileMeta &meta = sh.meta[n % kMetaStages], &next = sh.meta[(n + 1) % kMetaStages];
        const uint32_t st = n % kKvStages, dst = to0 + st * C::kStageBytes;
        if (n + 1 < tiles) ok = wait_bar(&sh.meta_full[(n + 1) % kMetaStages], ((n + 1) / kMetaStages) & 1) && ok;
        if (n >= (uint32_t)kKvStages) (void)wait_bar(&sh.kv_empty[st], ((n / kKvStages) - 1) & 1);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          uint32_t f[8];
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) e4m3x4_to_f16(w[e], f[2 * e], f[2 * e + 1]);
          const uint32_t factor = meta.factor[(row0 + i * kRowStep) >> p.own.log_bs];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = f16x2_mul(f[e], factor);
          const uint32_t at = dst + i * kRowStep * 128;
          st_shared(at + swz0, f[0], f[1], f[2], f[3]);
          st_shared(at + (swz0 ^ 16), f[4], f[5], f[6], f[7]);
          if (n + 1 < tiles) piece(next, i, raw[i]);  // on its way while this tile is used
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.kv_full[st]);
      }
    }
  } else {
    setmaxnreg_inc<kRegsSoft>();
    if (busy) {
      // ------------------------------------------------------------ softmax
      // A thread has a row from its q to its O.  Rows beyond the prefix's are zero in
      // Q: their results are not written.
      const int x = warp >> 2, row = tid & (kWG - 1);
      const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16), ocol = lane_addr + col_o(x);
      Walk walk = from;
      const uint32_t q_at = smem_u32(smem) + C::kOffQ + x * C::kStageBytes + row * 128;
      uint32_t n = 0;
      // A warp's rows of q on their way to shared memory, as they are: D / 8 lanes copy a
      // row's 16-byte pieces.
      auto load_q = [&](const Part &s) {
        constexpr int kLanes = D / 8;
        const int c = lane % kLanes;
#pragma unroll 4
        for (int i = 0; i < kLanes; ++i) {
          const int r = (warp & 3) * 32 + i * (32 / kLanes) + lane / kLanes;
          const bool there = x * kWG + r < s.rows;
          const uint32_t to = smem_u32(smem) + C::kOffQ + x * C::kStageBytes + (c >> 3) * kHalfTile + r * 128 + (((c & 7) ^ (r & 7)) << 4);
          cp_async_16(to, static_cast<const __nv_bfloat16 *>(p.own.q) + ((size_t)s.row0 + (there ? x * kWG + r : 0)) * D + c * 8, there ? 16 : 0);
        }
      };
      Part s = walk.next(sh.table, blockIdx.x);
      load_q(s);
#pragma unroll 1
      for (;;) {
        float m_run = -INFINITY, m_use = 0.f, l_run = 0.f;  // m_use: what is subtracted
        int unit = 0;
        const bool mine = x * kWG + row < s.rows;
        // bf16 -> fp16 with a factor for the row: the largest |q| becomes 224 .. 448;
        // a negative scale goes into q's sign
        float cs;
        {
          auto piece_at = [&](int c) { return q_at + (c >> 3) * kHalfTile + (((c & 7) ^ (row & 7)) << 4); };
          cp_async_wait();
          __syncwarp();
          uint32_t amax = 0;
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            uint32_t w[4];
            ld_shared(piece_at(c), w);
            amax = bf16x2_max(amax, bf16x2_max(bf16x2_max(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                               bf16x2_max(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu)));
          }
          const int ex = scale_exponent(__uint_as_float(max(amax & 0xffffu, amax >> 16) << 16), kLeastQExp);
          const float inv = p.own.scale < 0.f ? -exp2_int(-ex) : p.own.scale > 0.f ? exp2_int(-ex) : 0.f;
          cs = exp2_int(ex) * fabsf(p.own.scale) * 1.4426950408889634f;
          const uint64_t inv2 = f32x2(__float_as_uint(inv), __float_as_uint(inv));
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            uint32_t w[4];
            ld_shared(piece_at(c), w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo, hi;
              f32x2_split(fmul2(f32x2(w[e] << 16, w[e] & 0xffff0000u), inv2), lo, hi);
              w[e] = f16x2_rn(lo, hi);
            }
            st_shared(piece_at(c), w[0], w[1], w[2], w[3]);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.q_full[x]);
        }
#pragma unroll 1
        for (int j = s.j0; j < s.j1; ++j, ++n) {
          const int ms = n % kMetaStages;
          const TileMeta &meta = sh.meta[ms];
          (void)wait_bar(&sh.meta_full[ms], (n / kMetaStages) & 1);
          unit = meta.unit;
          const int odd = meta.odd, keys = meta.keys;
          if (meta.bad) l_run = __int_as_float(0x7fc00000);
          const float ck = fminf(fmaxf(cs * exp2_int(unit), FLT_MIN), FLT_MAX);
          const uint64_t ck2 = f32x2(__float_as_uint(ck), __float_as_uint(ck));
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            (void)wait_bar(&sh.s_full[x][h], n & 1);
            tc_fence_after();
            const uint32_t scol = lane_addr + col_s(x, 0) + h * 64;
            uint32_t sv[64];
            tmem_ld32(scol, *reinterpret_cast<uint32_t(*)[32]>(sv));
            tmem_ld32(scol + 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32));
            tmem_wait_ld();
            if (keys < kTileKeys) {
#pragma unroll
              for (int y = 0; y < 64; ++y)
                if (h * 64 + y >= keys) sv[y] = 0xff800000u;
            }
            if (odd) {
#pragma unroll
              for (int c = 0; c < 64; c += 16) {
                const float rest = meta.rest[(h * 64 + c) >> p.own.log_bs];
#pragma unroll
                for (int y = 0; y < 16; ++y) sv[c + y] = __float_as_uint(__uint_as_float(sv[c + y]) * rest);
              }
            }
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int y = 0; y < 64; y += 4) {
              m0 = fmax3(m0, __uint_as_float(sv[y]), __uint_as_float(sv[y + 1]));
              m1 = fmax3(m1, __uint_as_float(sv[y + 2]), __uint_as_float(sv[y + 3]));
            }
            const float mx = fmaxf(m0, m1) * ck;
            // raise the reference (seldom); the sums made with the old one follow
            const bool raise = mx > m_run + kRaiseLog2;  // at first: any key
            if (__any_sync(0xffffffffu, raise)) {
              const bool had = raise && m_run > -INFINITY;  // else O holds nothing of this row yet
              const float f = had ? ex2_approx(m_run - mx) : 1.f;
              l_run *= f;
              if (raise) m_run = mx;
              m_use = m_run == -INFINITY ? 0.f : m_run - kBias;
              if (__any_sync(0xffffffffu, had)) {
                (void)wait_bar(&sh.pv_done[x][h ^ 1], (h ? n : n - 1) & 1);
                tc_fence_after();
                scale_o<D>(ocol, f);
              }
            }
            const uint64_t nm2 = f32x2(__float_as_uint(-m_use), __float_as_uint(-m_use));
            uint64_t acc[2] = {0, 0};
            auto probabilities = [&](auto scaled) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int y = 0; y < 32; y += 2) {
                  float t0, t1;
                  f32x2_split(ffma2(f32x2(sv[32 * c + y], sv[32 * c + y + 1]), ck2, nm2), t0, t1);
                  float e0 = ex2_approx(t0), e1 = ex2_approx(t1);
                  acc[(y >> 1) & 1] = fadd2(acc[(y >> 1) & 1], f32x2(__float_as_uint(e0), __float_as_uint(e1)));
                  if constexpr (decltype(scaled)::value) {
                    const float rest = meta.rest[(h * 64 + 32 * c + y) >> p.own.log_bs];
                    e0 *= rest;
                    e1 *= rest;
                  }
                  pk[y >> 1] = f16x2_rn(e0, e1);
                }
                tmem_st16(scol + 16 * c, pk);
              }
            };
            if (odd) probabilities(std::true_type());
            else probabilities(std::false_type());
            float a, b;
            f32x2_split(fadd2(acc[0], acc[1]), a, b);
            l_run += a + b;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[x][h]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.meta_empty[ms]);
        }
        if (*abort_flag) l_run = __int_as_float(0x7fc00000);
        if (!s.last) {
          Walk ahead = walk;
          load_q(ahead.next(sh.table, blockIdx.x));  // arrives while O leaves
        }
        const bool merge = p.merge && s.whole;
        const int nrows = s.rows - x * kWG;
        const size_t at_row = merge ? (size_t)s.row0 + x * kWG : (size_t)s.slot * kRowTile + x * kWG;  // of the tile's first row
        float inv = exp2_int(unit) / l_run;
        if (merge) {
          // with the row's own part: (2^(lse - M) own + 2^(m - M) O) / (2^(lse - M) + 2^(m - M) l)
          const float m0 = mine ? p.own_lse[at_row + row] * 1.4426950408889634f : 0.f;
          const float M = fmaxf(m0, m_use), w0 = exp2f(m0 - M), w1 = exp2f(m_use - M), sum = fmaf(w1, l_run, w0);
          sh.own[x * kWG + row] = w0 / sum;
          inv = w1 * exp2_int(unit) / sum;
          if (mine) p.lse[at_row + row] = (M + log2f(sum)) * 0.69314718055994531f;
        } else if (mine) {
          p.part_ml[at_row + row] = make_float2(m_use, l_run);
        }
        (void)wait_bar(&sh.pv_done[x][1], (n - 1) & 1);
        tc_fence_after();
        // O leaves through shared memory, 64 bytes of a row at a time, so that four
        // lanes write a row's: a store to 32 rows takes 32 cycles.
        const uint32_t buf = smem_u32(sh.out) + x * kWG * 64, at = buf + row * 64, swz = (row >> 1) & 3;
        const int piece = lane & 3;
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          const size_t col = (size_t)(c * 16 + piece * 4);
          float4 own[4];
          if (merge) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = (warp & 3) * 32 + i * 8 + (lane >> 2);
              if (r < nrows) own[i] = *reinterpret_cast<const float4 *>(p.own_out + (at_row + r) * D + col);
            }
          }
          uint32_t o[16];
          tmem_ld16(ocol + c * 16, o);
          tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * inv);
#pragma unroll
          for (int y = 0; y < 4; ++y) st_shared(at + ((y ^ swz) << 4), o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = (warp & 3) * 32 + i * 8 + (lane >> 2);
            uint32_t v[4];
            ld_shared(buf + r * 64 + ((piece ^ ((r >> 1) & 3)) << 4), v);
            if (r >= nrows) continue;
            if (merge) {
              const float w0 = sh.own[x * kWG + r];
              const float4 u = own[i];
              *reinterpret_cast<uint2 *>(p.out + (at_row + r) * D + col) =
                  make_uint2(pack_bf16x2(fmaf(w0, u.x, __uint_as_float(v[0])), fmaf(w0, u.y, __uint_as_float(v[1]))),
                             pack_bf16x2(fmaf(w0, u.z, __uint_as_float(v[2])), fmaf(w0, u.w, __uint_as_float(v[3]))));
            } else {
              *reinterpret_cast<uint4 *>(p.part_o + (at_row + r) * D + col) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
          __syncwarp();
        }
        tc_fence_before();
        if (s.last) break;
        s = walk.next(sh.table, blockIdx.x);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sh.abort) atomicExch(status, HCA_ERR_TIMEOUT);
  if (warp == 15) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

// ---------------------------------------------------------------------------
// join: out = (w_0 o_0 + sum 2^(m_i - M) l_i o_i) / (w_0 + sum 2^(m_i - M) l_i) of a
// row's own keys (w_0 = 2^(lse - M)) and the parts of its prefix.  Bound by latency: table,
// references, parts, one after the other.  Of 643 row tiles 151 were cut in the case above:
// 25 us, 33 when the blocks looked at all tiles.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

// What a block's rows have of their own keys where a group's tiles were cut between
// CTAs (the combine kernel's work in hca_cache_attn).
struct OwnParts {
  int row, columns;  // rows of the group
  int slot0, cta;    // of the first part; the others have slots 2 (cta + i)
  int parts;
};

// What a join's block begins with.  All is loaded at once, and the block meets once.
struct JoinBegin {
  int units, quota, row_tiles;
  bool alone;    // some prefix has no common entries
  bool refused;  // then all rows are NaN, and written
};

template <int D, bool Own>
__device__ __forceinline__ JoinBegin join_begin(const SharedParams &p, Prefix *prefix) {
  constexpr int kLanes = D / 4, kRows = kJoinThreads / kLanes;
  constexpr uint32_t kLate = 1, kWrong = 2, kAlone = 4;
  static_assert(kSharedMaxGroups <= kJoinThreads, "a thread a prefix");
  __shared__ uint32_t seen[kJoinThreads / 32];
  const int tid = threadIdx.x;
  JoinBegin t = {p.table->units, p.table->quota, p.table->row_tiles, false, false};
  const int own_tiles = p.own.hdr->ntiles;
  uint32_t flags = 0;
  auto look = [&](int status) { flags |= status == HCA_ERR_TIMEOUT ? kLate | kWrong : status != HCA_OK ? kWrong : 0; };
  if constexpr (Own) {
    for (int i = tid; i < p.own.grid; i += kJoinThreads) look(p.own.err[i]);
  } else {
    look(p.own.hdr->status);
  }
  for (int i = tid; i < p.grid; i += kJoinThreads) look(p.err[i]);
  if (tid < p.own.G) {
    prefix[tid] = p.table->g[tid];
    if (prefix[tid].tiles == 0 && prefix[tid].rows > 0) flags |= kAlone;
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if ((tid & 31) == 0) seen[tid >> 5] = flags;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) flags |= seen[i];
  if (blockIdx.x == 0 && tid == 0) *p.status = flags & kLate ? HCA_ERR_TIMEOUT : flags & kWrong ? HCA_ERR_CACHE : HCA_OK;
  t.alone = flags & kAlone;
  t.refused = t.units < 0 || own_tiles < 0 || (flags & kLate);
  if (t.refused) {
    const size_t rows = (size_t)p.own.N * p.own.H;
    const int l = tid % kLanes;
    for (size_t row = (size_t)blockIdx.x * kRows + tid / kLanes; row < rows; row += (size_t)gridDim.x * kRows) {
      *reinterpret_cast<uint2 *>(p.out + row * D + 4 * l) = make_uint2(0x7fc07fc0u, 0x7fc07fc0u);
      if (l == 0) p.lse[row] = __int_as_float(0x7fc00000);
    }
  }
  return t;
}

__device__ __forceinline__ void add(float4 &o, float w, const float4 &v) {
  o.x = fmaf(w, v.x, o.x);
  o.y = fmaf(w, v.y, o.y);
  o.z = fmaf(w, v.z, o.z);
  o.w = fmaf(w, v.w, o.w);
}

// Few rows, many parts: a row has S groups of D / 4 lanes, each of which has every S-th
// part.  A lane looks at a part's reference and sum, and the first parts' O are on their way
// meanwhile.  With `Own` the parts of the requests' own keys are joined here too.  kBatch
// parts at a time: 8 where three blocks an SM are all there are, else 4 and more blocks
// (calls of 64 heads, columns of 64 entries: 4 tokens over 512 27.2 us and 28.5, 64 tokens
// over 390 62.5 and 60.0; with the parts' references one after the other 30.6 and 60.4).
// S is 4 where that many blocks run at once: 8 tokens of 8 heads over 65,536 entries 28.9
// us, 33.9 with 1 (25.6 since a CTA takes 8 steps at least).
template <int D, bool Own, int kBatch, int S>
__global__ void __launch_bounds__(kJoinThreads, kBatch == 8 ? 3 : 4) hca_cache_join_kernel(const SharedParams p) {
  constexpr int kLanes = D / 4, kRows = kJoinThreads / kLanes / S, kOwnBatch = 4;
  constexpr int kChunks = kRowTile / kRows;  // of a row tile, a block's each
  constexpr float kLog2e = 1.4426950408889634f;
  __shared__ Prefix prefix[kSharedMaxGroups];
  __shared__ OwnParts cut[kRows];  // a block's rows have as many groups at most
  __shared__ int ncut;
  __shared__ float4 group_o[S > 1 ? kJoinThreads : 1];
  __shared__ float2 group_ml[S > 1 ? kJoinThreads / kLanes : 1];
  const int tid = threadIdx.x, l = tid % kLanes, lane0 = (tid & 31) & ~(kLanes - 1), group = tid / kLanes, h = group / kRows;
  pdl_wait();
  Border border[2];  // of two of the own keys' CTAs, of which there are 2 kMaxGrid at most
  if constexpr (Own) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      border[i] = Border{0, 0, 0, 0};
      if (tid + i * kJoinThreads < p.own.grid) border[i] = p.own.border[tid + i * kJoinThreads];
    }
    if (tid == 0) ncut = 0;
  }
  static_assert(kMaxGrid <= kJoinThreads, "a thread has the borders of two CTAs");
  const JoinBegin t = join_begin<D, Own>(p, prefix);
  if (t.refused) return;
  const int quota = t.quota, items = t.row_tiles * kChunks;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    int lo = 0, hi = p.own.G;  // the row tile's prefix
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid].rt0 <= item / kChunks) lo = mid; else hi = mid;
    }
    const Prefix x = prefix[lo];
    const int rt = item / kChunks - x.rt0, u0 = x.line0 + rt * x.span, first = u0 / quota;
    const int r0 = item % kChunks * kRows + group % kRows, r = rt * kRowTile + r0;  // of the tile, of the prefix
    const size_t row = (size_t)x.row0 + r;
    const bool there = r < x.rows;
    const int parts = there && x.tiles > 0 ? (u0 + x.span - 1) / quota - first + 1 : 0;
    const int n = (parts - h + S - 1) / S;                                          // of the group: h, h + S, ...
    const size_t slot = (size_t)(x.rt0 + rt + first + h) * kRowTile + r0, step = S * kRowTile;  // of them, from one to the next
    const float *part = p.part_o + slot * D + 4 * l;
    float4 v[kBatch];
    auto load = [&](int i) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        v[k] = i + k < n ? *reinterpret_cast<const float4 *>(part + (i + k) * step * D) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);
    auto ml_of = [&](int i) { return i < n ? p.part_ml[slot + i * step] : make_float2(-INFINITY, 0.f); };
    const float2 ml0 = ml_of(l);
    OwnParts mine = {0, 0, 0, 0, 0};
    if constexpr (Own) {
      // the groups among the block's rows that were cut
      const int a = x.row0 + rt * kRowTile + item % kChunks * kRows, e = min(a + kRows, x.row0 + x.rows);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Border b = border[i];
        if (b.columns > 0 && b.row < e && b.row + b.columns > a)
          cut[atomicAdd(&ncut, 1)] = OwnParts{b.row, b.columns, b.slot, tid + i * kJoinThreads, b.parts};
      }
      __syncthreads();
      for (int i = 0; there && i < ncut; ++i)
        if ((int)row >= cut[i].row && (int)row < cut[i].row + cut[i].columns) mine = cut[i];
      if (item + (int)gridDim.x < items) {
        __syncthreads();
        if (tid == 0) ncut = 0;
        __syncthreads();
      }
    }
    const bool joined = parts > 0 || mine.parts > 0;
    const int m = h == S - 1 ? mine.parts : 0;                      // parts of the row's own keys: the last group's
    const bool whole = there && h == S - 1 && mine.parts == 0;  // these are in own_out
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float lse = 0.f;
    if (whole) {
      o = *reinterpret_cast<const float4 *>(p.own_out + row * D + 4 * l);
      lse = p.own_lse[row];
    }
    auto own_slot = [&](int i) { return i == 0 ? mine.slot0 : 2 * (mine.cta + i); };
    auto own_at = [&](int i) { return (size_t)own_slot(i) * p.own.NQ + ((int)row - mine.row); };
    auto own_ml_of = [&](int i) { return i < m ? p.own.part_ml[own_at(i)] : make_float2(-INFINITY, 0.f); };
    // the group's greatest reference
    float M = whole ? lse * kLog2e : -INFINITY;
    for (int i = l; i < n; i += kLanes) M = fmaxf(M, i == l ? ml0.x : ml_of(i).x);
    for (int i = l; i < m; i += kLanes) M = fmaxf(M, own_ml_of(i).x);
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    const float w0 = whole ? joined ? exp2f(lse * kLog2e - M) : 1.f : 0.f;
    o.x *= w0; o.y *= w0; o.z *= w0; o.w *= w0;
    float sum = l == 0 ? w0 : 0.f;  // a lane's parts
    // The rows of a warp may have different numbers of parts: its loops are the longest's.
    const int most = __reduce_max_sync(0xffffffffu, n), own_most = Own ? __reduce_max_sync(0xffffffffu, m) : 0;
    for (int c = 0; c < own_most; c += kLanes) {
      const float2 ml = own_ml_of(c + l);
      // O / l as the prefixes' parts have it: 2^unit / l is a normal number; l = 0: a part in which the row saw no key
      const float w = ml.y != 0.f ? exp2f(ml.x - M) * ml.y : 0.f;
      const float f = w != 0.f ? w * (exp2_int(p.own.part_unit[own_slot(c + l)]) / ml.y) : 0.f;
      sum += w;
#pragma unroll 1
      for (int i = 0; i < min(kLanes, own_most - c); i += kOwnBatch) {
        float fs[kOwnBatch];
        float4 u[kOwnBatch];
#pragma unroll
        for (int k = 0; k < kOwnBatch; ++k) {
          fs[k] = __shfl_sync(0xffffffffu, f, lane0 + i + k);
          u[k] = fs[k] != 0.f ? *reinterpret_cast<const float4 *>(p.own.part_o + own_at(c + i + k) * D + 4 * l) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kOwnBatch; ++k) add(o, fs[k], u[k]);
      }
    }
    for (int c = 0; c < most; c += kLanes) {
      const float2 ml = c == 0 ? ml0 : ml_of(c + l);
      const float w = c + l < n ? exp2f(ml.x - M) * ml.y : 0.f;
      sum += w;
#pragma unroll 1
      for (int i = 0; i < min(kLanes, most - c); i += kBatch) {
        if (c + i > 0) load(c + i);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) add(o, __shfl_sync(0xffffffffu, w, lane0 + i + k), v[k]);
      }
    }
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if constexpr (S > 1) {
      // the row's groups
      group_o[tid] = o;
      if (l == 0) group_ml[group] = make_float2(M, sum);
      __syncthreads();
      if (h == S - 1) {
        const int of = group % kRows;
        for (int i = 0; i < S - 1; ++i) M = fmaxf(M, group_ml[of + i * kRows].x);
        float2 ml = group_ml[group];
        const float f = joined ? exp2f(ml.x - M) : 1.f;
        sum = f * ml.y;
        o.x *= f; o.y *= f; o.z *= f; o.w *= f;
        for (int i = 0; i < S - 1; ++i) {
          ml = group_ml[of + i * kRows];
          const float w = ml.x > -INFINITY ? exp2f(ml.x - M) : 0.f;  // no part: not minus infinity less itself
          sum = fmaf(w, ml.y, sum);
          add(o, w, group_o[(of + i * kRows) * kLanes + l]);
        }
      }
      __syncthreads();
    }
    if (!there || h != S - 1) continue;
    const float inv = joined ? 1.f / sum : 1.f;
    *reinterpret_cast<uint2 *>(p.out + row * D + 4 * l) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (l == 0) p.lse[row] = joined ? (M + log2f(sum)) * 0.69314718055994531f : lse;
  }
}

// Many rows, of which whole row tiles were finished by the CTA that had them: those in
// which a CTA's range begins (the first that does) and those without common entries.
// A lane has U rows at a time, whose loads are in flight together.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) hca_cache_join_many_kernel(const SharedParams p) {
  constexpr int U = 4, kLanes = D / 4, kRows = kJoinThreads / kLanes;
  constexpr int kChunks = kRowTile / (kRows * U);  // of a row tile, a block's each
  constexpr float kLog2e = 1.4426950408889634f;
  __shared__ Prefix prefix[kSharedMaxGroups];
  const int tid = threadIdx.x, l = tid % kLanes;
  pdl_wait();
  const JoinBegin t = join_begin<D, false>(p, prefix);
  if (t.refused) return;
  const int units = t.units, quota = t.quota;
  const int begins = p.grid * kChunks, items = begins + (t.alone ? t.row_tiles * kChunks : 0);
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int tile = (item < begins ? item : item - begins) / kChunks;
    const long long u = (long long)tile * quota;
    if (item < begins && u >= units) continue;
    int lo = 0, hi = p.own.G;  // the row tile's prefix
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (item < begins ? prefix[mid].line0 <= u : prefix[mid].rt0 <= tile) lo = mid; else hi = mid;
    }
    const Prefix x = prefix[lo];
    if (item >= begins && x.tiles > 0) continue;
    const int rt = item < begins ? ((int)u - x.line0) / x.span : tile - x.rt0, u0 = x.line0 + rt * x.span, first = u0 / quota;
    if (item < begins && (u0 == u || u - quota > u0)) continue;
    const int parts = x.tiles > 0 ? (u0 + x.span - 1) / quota - first + 1 : 0;
    const int r0 = item % kChunks * (kRows * U) + tid / kLanes;  // the lane's first row; the others are kRows apart
    float4 o[U];
    float lse[U], M[U], sum[U];
    size_t slot[U];
    bool there[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = rt * kRowTile + r0 + i * kRows;
      there[i] = r < x.rows;
      slot[i] = (size_t)(x.rt0 + rt + first) * kRowTile + r0 + i * kRows;  // the next part's is 256 further
      o[i] = there[i] ? *reinterpret_cast<const float4 *>(p.own_out + (size_t)(x.row0 + r) * D + 4 * l) : make_float4(0.f, 0.f, 0.f, 0.f);
      lse[i] = there[i] ? p.own_lse[x.row0 + r] : 0.f;
      M[i] = lse[i] * kLog2e;
    }
    for (int k = 0; k < parts; ++k) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (there[i]) M[i] = fmaxf(M[i], p.part_ml[slot[i] + (size_t)k * kRowTile].x);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      sum[i] = parts > 0 ? exp2f(lse[i] * kLog2e - M[i]) : 1.f;
      o[i].x *= sum[i]; o[i].y *= sum[i]; o[i].z *= sum[i]; o[i].w *= sum[i];
    }
#pragma unroll 1
    for (int k = 0; k < parts; ++k) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (!there[i]) continue;
        const size_t at = slot[i] + (size_t)k * kRowTile;
        const float2 ml = p.part_ml[at];
        const float w = exp2f(ml.x - M[i]) * ml.y;
        sum[i] += w;
        add(o[i], w, *reinterpret_cast<const float4 *>(p.part_o + at * D + 4 * l));
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (!there[i]) continue;
      const size_t row = (size_t)x.row0 + rt * kRowTile + r0 + i * kRows;
      const float inv = parts > 0 ? 1.f / sum[i] : 1.f;
      *reinterpret_cast<uint2 *>(p.out + row * D + 4 * l) = make_uint2(pack_bf16x2(o[i].x * inv, o[i].y * inv), pack_bf16x2(o[i].z * inv, o[i].w * inv));
      if (l == 0) p.lse[row] = parts > 0 ? (M[i] + log2f(sum[i])) * 0.69314718055994531f : lse[i];
    }
  }
}

struct Layout {
  size_t off_table, off_own, off_out, off_lse, off_err, off_ml, off_o, bytes;
};

Layout layout_of(int N, int R, int H, int D, int G) {
  Layout l;
  const size_t rows = (size_t)N * H, slots = rows / kRowTile + G + kMaxGrid;
  size_t at = kHeaderBytes;
  l.off_table = at;
  at += align_up(sizeof(Table));
  l.off_own = at;
  at += align_up(cache_attn_ws_bytes(N, R, H, D, HCA_BF16));
  l.off_out = at;
  at += align_up(rows * D * sizeof(float));
  l.off_lse = at;
  at += align_up(rows * sizeof(float));
  l.off_err = at;
  at += align_up(kMaxGrid * sizeof(int32_t));
  l.off_ml = at;
  at += align_up(slots * kRowTile * sizeof(float2));
  l.off_o = at;
  at += align_up(slots * kRowTile * D * sizeof(float));
  l.bytes = at;
  return l;
}

template <int D>
cudaError_t launch(const CacheAttnArgs &a, SharedParams &p, int sms, cudaStream_t st) {
  using C = Cfg<D>;
  static SmemAttrOnce attr;
  cudaError_t e = attr.ensure(reinterpret_cast<const void *>(hca_cache_prefix_kernel<D>), C::kSmem);
  if (e != cudaSuccess) return e;
  auto prefix = [&] {
    ProfScope prof(kKCachePrefix, st);
    hca_cache_prefix_kernel<D><<<p.grid, kThreads, C::kSmem, st>>>(p);
    return cudaGetLastError();
  };
  if (!p.merge) e = prefix();
  if (e == cudaSuccess) e = cache_attn(a, st);
  if (e == cudaSuccess && p.merge) e = prefix();
  if (e != cudaSuccess) return e;
  ProfScope prof(kKCacheJoin, st);
  auto join = [&](auto *kernel, long long rows, long long most) {  // of a block, blocks
    const long long blocks = (long long)p.own.N * p.own.H / rows + p.own.G * (kRowTile / rows);
    return launch_behind(kernel, dim3((unsigned)std::min(blocks, most)), kJoinThreads, 0, st, p);
  };
  constexpr int kRows = kJoinThreads / (D / 4);
  if (p.merge) return join(hca_cache_join_many_kernel<D>, 4 * kRows, 3 * sms);
  if (!p.own.joined) return join(hca_cache_join_kernel<D, false, 4, 1>, kRows, 5 * sms);
  const long long blocks = (long long)p.own.N * p.own.H / kRows;
  if (4 * blocks <= 3 * sms) return join(hca_cache_join_kernel<D, true, 8, 4>, kRows / 4, 3 * sms);
  if (blocks <= 3 * sms) return join(hca_cache_join_kernel<D, true, 8, 1>, kRows, 3 * sms);
  return join(hca_cache_join_kernel<D, true, 4, 1>, kRows, 5 * sms);
}

}  // namespace

int cache_shared_max_groups() { return kSharedMaxGroups; }

size_t cache_attn_shared_ws_bytes(int N, int R, int H, int D, int G, int dtype) {
  return dtype == HCA_F32 ? cache_attn_ws_bytes(N, R, H, D, dtype) : layout_of(N, R, H, D, G).bytes;
}

namespace {

// Is it worth attending the common entries apart?  Of the lengths the host knows how many
// rows and prefixes there are and how many key tiles the compressed tables hold at most:
// it takes that for the common length, and the rows for shared out evenly among the
// prefixes, whose row tiles are their own.  In us, with `groups` of rows that share key tiles where nothing else is shared, of
// 128 rows or fewer, on 152 SMs:
//   by itself  19 + groups (tiles + 6) / 304 * 1.7 (2.0 for groups of 128 rows) + what the
//              parts of a group take to join
//   apart      22 + steps of a CTA * 1.5 + groups * 8 / 152 * 1.2 + rows to join
// Measured (64 heads, D = 128, by themselves | apart): 64 tokens over 8 tiles 23 | 28,
// 64 tiles 47 | 38, 512 tiles 203 | 105; 16 tokens over 64 tiles 26 | 27, 512 tiles 69 |
// 44; 4 tokens over 64 tiles 22 | 25, 512 tiles 37 | 32; 1 token over 128 tiles 21 | 24, 512
// 36 | 29; 200 tokens over 16 tiles 45 | 48, 256 tiles 305 | 167; 8 heads, 64 tokens over 16
// tiles 25 | 27, 512 tiles 197 | 35; 314 prompt tokens over 32 tiles 66 | 73, 256 tiles
// 293 | 237.  As many prefixes, 64 heads, 64 tokens over 132 tiles: 16 prefixes 70 | 47, 64
// prefixes 71 | 117; 64 over 516 tiles 209 | 347.  D = 64: 64 tokens over 28 tiles 26 | 29, 68
// tiles 39 | 32; 64 prefixes over 68 tiles 39 | 65.  Of 264 calls (1 to 541 tokens of 1 to
// 200 prefixes, 8 to 128 heads, both D, 12 to 516 tiles) the rule took the slower way in 7
// by 5% or more, the worst by 21% (541 tokens of 6 prefixes over 132 tiles 267 | 323).
bool apart_pays(const CacheAttnArgs &a, int sms) {
  const double groups = std::max(1.0, (double)cache_attn_groups(a.N, a.R, a.H, a.D, a.dtype));
  const double rows = (double)a.N * a.H, full = rows >= 100.0 * groups ? 2.0 : 1.7, tiles = std::min((double)a.comp.cols * a.bs / kTileKeys, 8388608.0);
  const double alone = 19 + groups * (tiles + 6) / (2.0 * sms) * full + 0.08 * std::min(tiles / 2, 2.0 * sms / groups);
  const double prefixes = std::max(1, std::min({a.share.G, a.R, a.N}));
  const double steps = std::max(prefixes * std::ceil(rows / (kRowTile * prefixes)) * tiles / sms, std::sqrt(tiles / 8));
  const double apart = 22 + steps * 1.5 + groups * 8 / sms * 1.2 + rows * 0.0007;
  return apart < alone;
}

}  // namespace

cudaError_t cache_attn_shared(const CacheAttnArgs &args, cudaStream_t st) {
  CacheAttnArgs a = args;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorNoDevice;
  const int path = shared_path_setting();
  // fp32: the kernel has no groups across requests, so each attends the common entries with
  // its own (64 requests of 4 heads, D = 64, over 512 common tiles 300 us, one of them 37)
  if (a.dtype == HCA_F32 || path == 2 || (path == 0 && !apart_pays(a, sms))) {
    a.share.apart = 0;
    return cache_attn(a, st);
  }
  const Layout l = layout_of(a.N, a.R, a.H, a.D, a.share.G);
  char *ws = static_cast<char *>(a.ws);
  SharedParams p;
  p.table = reinterpret_cast<Table *>(ws + l.off_table);
  p.err = reinterpret_cast<int32_t *>(ws + l.off_err);
  p.part_ml = reinterpret_cast<float2 *>(ws + l.off_ml);
  p.part_o = reinterpret_cast<float *>(ws + l.off_o);
  p.own_out = reinterpret_cast<const float *>(ws + l.off_out);
  p.own_lse = reinterpret_cast<const float *>(ws + l.off_lse);
  p.status = reinterpret_cast<int32_t *>(ws);
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  p.grid = std::min(sms, kMaxGrid);
  // As many row tiles as CTAs: most are one CTA's, which adds the rows' own part
  // where it has O.  Otherwise both run at the same time.
  p.merge = (long long)a.N * a.H >= (long long)kRowTile * p.grid;
  p.stall = a.stall;
  a.stall = 0;
  a.out = ws + l.off_out;
  a.lse = reinterpret_cast<float *>(ws + l.off_lse);
  a.ws = ws + l.off_own;
  a.share.apart = 1;
  a.share.beside = !p.merge && sms <= kMaxGrid;
  // The parts of the own keys in the same launch, where each block has one item (4,096
  // rows over 24,960 entries 60 us, 69 with a launch of their own); with more items a
  // block it is slower (12,800 rows over 4,096 entries 60 us, 57).
  a.share.joined = (long long)a.N * a.H * (a.D / 4) <= 5ll * sms * kJoinThreads;
  shared_params(a, p.own);
  return a.D == 64 ? launch<64>(a, p, sms, st) : launch<128>(a, p, sms, st);
}

}  // namespace hca
