// hca_cache_attn.cuh -- parameters of the attention-over-cache kernels.
#pragma once

#include <climits>

#include "hca_cache.cuh"

namespace hca {
namespace cache {

// CTAs of a launch, at most (the workspace holds two partial results for each)
inline int max_ctas(bool tensor_cores) { return tensor_cores ? 320 : 640; }
constexpr int kSimtCols = 16;   // columns of an fp32 group

struct AttnParams {
  const void *q;
  const int32_t *start, *held;
  CacheSet raw, comp;
  void *out;
  float *lse;
  SchedHeader *hdr;
  Group *groups;
  int32_t *gbase;      // [R + 1] first group (before slicing) of each request
  int32_t *err;        // [grid] status of each CTA
  Border *border;      // [grid]
  float2 *part_ml;     // [2 * grid][NQ] reference exponent and sum of a partial result
  float *part_o;       // [2 * grid][NQ][D], in units of 2^part_unit
  int32_t *part_unit;  // [2 * grid]
  int N, R, H, D, W, m, log_bs;
  int HS, slices, P;   // heads per slice, slices, positions per group
  int NQ;              // columns of a group, P * HS <= NQ
  int grid;            // CTAs of the attention kernel
  int min_tiles;       // fewest tiles of a CTA
  int in_cta;          // the attention kernel's CTAs work out the schedule themselves
  float scale;
  uint64_t wait_ns;
  int stall;
  static constexpr bool kShared = false;
};

// The requests of prefix g are first[g] .. first[g + 1] - 1; the first cols[g]
// columns of their compressed tables are the same blocks.
struct SharedAttnParams : AttnParams {
  const int32_t *first, *cols;
  int G;
  int apart;  // those columns are left out, and out is fp32 (the join adds them)
  int beside; // the kernel of the prefixes runs at the same time, on other SMs
  int joined; // the join of the prefixes has the parts of these keys too
  int sms;
  static constexpr bool kShared = true;
};

// Prefixes are in order and cover all requests (each thread of a block looks at its
// own of them).
__device__ __forceinline__ bool prefixes_ok(const AttnParams &) { return true; }
__device__ __forceinline__ bool prefixes_ok(const SharedAttnParams &p) {
  bool ok = true;
  for (int g = threadIdx.x; g < p.G; g += blockDim.x)
    ok = ok && p.first[g] <= p.first[g + 1] && p.cols[g] >= 0 && p.cols[g] <= p.comp.cols && (g > 0 || p.first[0] == 0) &&
         (g < p.G - 1 || p.first[p.G] == p.R);
  return ok;
}

// Common columns of request r's prefix
__device__ __forceinline__ int prefix_pages(const AttnParams &, int) { return 0; }
__device__ __forceinline__ int prefix_pages(const SharedAttnParams &p, int r) {
  int lo = 0, hi = p.G;  // first[lo] <= r < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.first[mid] <= r) lo = mid; else hi = mid;
  }
  return p.cols[lo];
}

// What of a group's pages is not its prefix's
__device__ __forceinline__ Pages own_pages(const AttnParams &, int, const Pages &pg) { return pg; }
__device__ __forceinline__ Pages own_pages(const SharedAttnParams &p, int r, Pages pg) {
  if (p.apart) {
    pg.cp0 = prefix_pages(p, r);
    pg.ncomp -= pg.cp0;
  }
  return pg;
}

__device__ __forceinline__ bool wide_rows(const AttnParams &) { return false; }
__device__ __forceinline__ bool wide_rows(const SharedAttnParams &p) { return p.apart != 0; }

// Columns of a group that stand for a (position, head).
__device__ __forceinline__ int real_columns(const AttnParams &p, int npos, int slice) {
  return p.P == 1 ? min(p.HS, p.H - slice * p.HS) : npos * p.HS;
}

// Tiles [c0, c1) of the line and what of group g lies in them.
__device__ __forceinline__ Segment segment_of(const Group &g, int c0, int c1, int cta) {
  Segment s;
  const int a = max(g.tile0, c0), b = min(g.tile0 + g.ntiles, c1);
  s.r = g.r; s.row0 = g.row0; s.pos0 = g.pos0; s.npos = g.npos;
  s.j0 = a - g.tile0;
  s.j1 = b - g.tile0;
  // the group that enters the CTA's range from before it takes slot 0
  s.slot = s.j0 == 0 && s.j1 == g.ntiles ? -1 : 2 * cta + (a == c0 ? 0 : 1);
  s.slice_last = 2 * g.slice + (b == c1 ? 1 : 0);
  return s;
}

// The join at the end of this CTA's range, if its last group begins in it.
__device__ __forceinline__ Border border_of(const AttnParams &p, const Group &g, int c0, int c1, int quota, int cta) {
  Border x = {0, 0, 0, 0};
  const int end = g.tile0 + g.ntiles;
  if (g.tile0 >= c0 && end > c1) {
    x.row = g.row0 * p.H + g.slice * p.HS;
    x.columns = real_columns(p, g.npos, g.slice);
    x.parts = (end - 1) / quota - cta + 1;
    x.slot = 2 * cta + (g.tile0 == c0 ? 0 : 1);
  }
  return x;
}

// Chunks (groups before slicing) of request r; false: lengths out of range.
template <typename P>
__device__ __forceinline__ bool request_chunks(const P &p, int r, int &n) {
  const int s0 = p.start[r], s1 = p.start[r + 1], h = p.held[r];
  bool ok = s0 >= 0 && s1 >= s0 && s1 <= p.N && h >= 0 && h <= kMaxPos - (s1 - s0) && (r > 0 || s0 == 0);
  if constexpr (P::kShared) {
    // every token sees the whole prefix
    const long long c = prefix_pages(p, r);
    ok = ok && c >= 0 && c <= p.comp.cols && (s1 == s0 || (c << p.log_bs) * p.m <= (long long)h + 1);
  }
  n = ok ? (s1 - s0 + p.P - 1) / p.P : 0;
  return ok;
}

// Group of chunk c, the k-th of request r; false: the tables are too narrow.
template <typename P>
__device__ __forceinline__ bool chunk_group(const P &p, int r, int k, Group &g) {
  const int s0 = p.start[r], T = p.start[r + 1] - s0, h = p.held[r], first = k * p.P;
  g.r = r;
  g.row0 = s0 + first;
  g.pos0 = h + first;
  g.npos = min(p.P, T - first);
  g.slice = 0;
  const Pages pg = own_pages(p, r, group_pages(g.pos0, g.npos, p.W, p.m, p.log_bs, p.comp.table != nullptr));
  g.ntiles = (int)((((uint32_t)(pg.nraw + pg.ncomp) << p.log_bs) + kTileKeys - 1) / kTileKeys);
  // the raw table keeps the last cols pages of the request's tokens
  return ((h + T - 1) >> p.log_bs) - pg.rp0 < p.raw.cols && pg.cp0 + pg.ncomp <= p.comp.cols;
}

// Rows of a prefix that share the converted keys on an SM, and a step of theirs is 128
// keys (hca_cache_shared.cu).
constexpr int kRowTile = 256;

// A prefix's rows and key tiles; false: it does not fit.
struct PrefixSize {
  int row0, rows, tiles;
  __device__ __forceinline__ int row_tiles() const { return (rows + kRowTile - 1) / kRowTile; }
};
__device__ __forceinline__ bool prefix_size(const SharedAttnParams &p, int g, PrefixSize &x) {
  x = PrefixSize{0, 0, 0};
  const int f0 = p.first[g], f1 = p.first[g + 1], c = p.cols[g];
  if (f0 < 0 || f1 < f0 || f1 > p.R || (g == 0 && f0 != 0) || (g == p.G - 1 && f1 != p.R) || c < 0 || c > p.comp.cols ||
      ((long long)c << p.log_bs) > kMaxPos)
    return false;
  const int s0 = p.start[f0], s1 = p.start[f1];
  if (s0 < 0 || s1 < s0 || s1 > p.N) return false;
  x.row0 = s0 * p.H;
  x.rows = (s1 - s0) * p.H;
  x.tiles = ((c << p.log_bs) + kTileKeys - 1) / kTileKeys;
  return true;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Tiles of the requests' own keys, those of requests i, i + step, ...: each is
// estimated by its last chunk's.
__device__ __forceinline__ long long own_tiles(const SharedAttnParams &p, int i, int step) {
  long long own = 0;
  for (int r = i; r < p.R; r += step) {
    int n;
    Group g;
    g.ntiles = 0;
    if (request_chunks(p, r, n) && n > 0) (void)chunk_group(p, r, n - 1, g);
    own += (long long)(g.ntiles + kGroupCost) * n * p.slices;
  }
  return own;
}

// SMs of the prefixes' kernel, when it has `units` steps in all and the requests'
// own keys (`own` tiles) run beside it: so many that both end at about the same time
// (all lanes of a warp call it).  A step takes 1.65 us, an own tile 2.8 us with two
// CTAs on an SM (a group's beginning and end two more).  What the two kernels make
// of it need not agree.
__device__ __forceinline__ int prefix_sms(const SharedAttnParams &p, long long units, long long own) {
  if (units == 0) return 0;
  float best = INFINITY;
  int at = 1;
  for (int s = 1 + (threadIdx.x & 31); s < p.sms; s += 32) {  // SMs of the own keys
    const float a = ceilf(__fdividef((float)units, (float)(p.sms - s))) * 1.65f;
    const float b = fmaxf(ceilf(__fdividef((float)own, (float)(2 * s))), (float)p.min_tiles) * 2.8f;
    const float t = fmaxf(a, b);
    if (t < best) best = t, at = s;
  }
  const uint32_t least = __reduce_min_sync(0xffffffffu, __float_as_uint(best));  // positive floats are in order
  at = __reduce_min_sync(0xffffffffu, __float_as_uint(best) == least ? at : INT_MAX);
  return p.sms - at;
}

// CTAs that the own keys' kernel works with (`tmp` holds 33 values)
__device__ __forceinline__ int own_grid(const AttnParams &p, long long *) { return p.grid; }
__device__ __forceinline__ int own_grid(const SharedAttnParams &p, long long *tmp) {
  if (!p.beside) return p.grid;
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  PrefixSize x = {0, 0, 0};
  if ((int)threadIdx.x < p.G) (void)prefix_size(p, threadIdx.x, x);
  const long long u = warp_sum((long long)x.row_tiles() * x.tiles), o = warp_sum(own_tiles(p, threadIdx.x, blockDim.x));
  if ((threadIdx.x & 31) == 0) {
    tmp[warp] = u;
    tmp[16 + warp] = o;
  }
  __syncthreads();
  long long units = 0, own = 0;
  for (int w = 0; w < warps; ++w) {
    units += tmp[w];
    own += tmp[16 + w];
  }
  return min(p.grid, 2 * (p.sms - prefix_sms(p, units, own)));
}

// what of a call the kernels get (hca_cache_attn.cu)
void shared_params(const CacheAttnArgs &a, SharedAttnParams &p);

// tensor-core kernel (hca_cache_attn_tc.cu)
int tc_cache_ctas();     // CTAs per SM
int tc_cache_threads();  // threads of a CTA
cudaError_t tc_cache_attn(const AttnParams &p, cudaStream_t st);
cudaError_t tc_cache_attn(const SharedAttnParams &p, cudaStream_t st);

}  // namespace cache
}  // namespace hca
